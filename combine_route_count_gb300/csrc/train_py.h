// The methods of the CPython module _ffn that train_py.cc has.
#pragma once

#include <Python.h>

PyMethodDef* train_methods();
