"""The feed-forward calls on tensors launch without the interpreter lock.

A child process loads _ffn beside a stand-in for libmoe.so whose entry points
answer whether their thread holds the lock.  (Tensors on a GPU are needed for the argument
checks before the call; nothing is launched.)"""
import os
import subprocess
import sys
import sysconfig

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

STUB = """
#include <Python.h>
// 1: the calling thread holds the interpreter lock (MOE_EINVAL for the caller), 0: not.
#define ANSWER(name) extern "C" int name() { return PyGILState_Check(); }
ANSWER(moe_add_rms_norm_fp8) ANSWER(moe_expert_gemm_fp8) ANSWER(moe_expert_glu_fp8) ANSWER(moe_decode_layer_fp8)
extern "C" int stub_is_loaded() { return PyGILState_Check(); }
"""

CHILD = """
import ctypes, importlib.util, struct, sys
import torch
stub = ctypes.PyDLL(sys.argv[1] + "/libmoe.so")
assert stub.stub_is_loaded() == 1  # the answer with the lock
spec = importlib.util.spec_from_file_location("_ffn", sys.argv[1] + "/_ffn.so")
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)

class Error(Exception):
    pass

m.init(Error)
u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
f32 = lambda *s: torch.zeros(s, device="cuda")
bf16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
m.add_rms_norm_fp8(bf16(2, 256), f32(256), u8(2, 256), f32(2, 2), 1e-6, None, None, None, 0)
m.expert_product(False, u8(2, 256), f32(2, 2), u8(256, 256), f32(2, 2), f32(2, 256), None, None, None, 0)
m.expert_product(True, u8(2, 256), f32(2, 2), u8(256, 256), f32(2, 2), u8(2, 128), f32(2, 1), None, None, 0)
plan = struct.pack("6i3Q", 4, 256, 2, 8, 128, 0, 0, 0, 0)
weights = (u8(8, 256, 256), f32(8, 2, 2), u8(8, 256, 128), f32(8, 2, 1))
m.decode_layer_fp8(plan, weights, u8(2, 256), f32(2, 2), i32(2, 2), f32(2, 2), bf16(2, 256), 0)
print("four calls without the lock")
"""


def test_no_lock_in_a_launch(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_route_count_gb300 import build
    build.build_ffn()
    (tmp_path / "stub.cc").write_text(STUB)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-fPIC", "-shared", "-Wl,-soname,libmoe.so",
                    "-I", sysconfig.get_paths()["include"], str(tmp_path / "stub.cc"), "-o", str(tmp_path / "libmoe.so")],
                   check=True)
    os.symlink(build.LIB_FFN, tmp_path / "_ffn.so")
    r = subprocess.run([sys.executable, "-c", CHILD, str(tmp_path)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "without the lock" in r.stdout, r.stdout + r.stderr


def in_a_new_thread(f):
    import threading
    result = []

    def work():
        try:
            result.append(f())
        except Exception as e:  # noqa: BLE001
            result.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not isinstance(result[0], Exception), result[0]


def test_a_thread_whose_first_cuda_call_is_a_product():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_decode_layer import run, tokens, weights
    from test_gpu_expert_gemm import inputs, offsets_of

    from combine_route_count_gb300 import build, ffn
    build.build_ffn()
    # The few-row kernel, row groups and the tile kernel; then the layer.
    for counts, N, K in (([7], 136, 128), ([2] * 12, 264, 40 * 128), ([300, 100], 512, 1024)):
        args, off = inputs(1, sum(counts), len(counts), N, K), offsets_of(counts) if len(counts) > 1 else None
        want, out = torch.empty(sum(counts), N, device="cuda"), torch.zeros(sum(counts), N, device="cuda")
        ffn.expert_gemm_fp8(*args, want, expert_offsets=off)
        torch.cuda.synchronize()
        in_a_new_thread(lambda: ffn.expert_gemm_fp8(*args, out, expert_offsets=off, stream=0))
        assert torch.equal(out, want)
    tk = tokens(2, 6, 256, 2, 8)
    layer = ffn.DecodeLayer(6, 2, *weights(1, 8, 256, 128))
    want, out = run(layer, *tk), torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
    in_a_new_thread(lambda: layer.forward(*tk, out, stream=0))
    assert torch.equal(out, want)


@pytest.mark.parametrize("threads", [2, 4])
def test_one_layer_from_several_threads(threads):
    """Calls of several threads on one stream come one after the other, both kernels of each together."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import threading

    from test_gpu_decode_layer import run, tokens, weights

    from combine_route_count_gb300 import build, ffn
    build.build_ffn()
    layer = ffn.DecodeLayer(16, 4, *weights(1, 16, 512, 384))
    batches = [tokens(2 + i, 16 - i, 512, 4, 16) for i in range(threads)]
    alone = [run(layer, *b) for b in batches]
    outs = [torch.zeros(400, *a.shape, dtype=a.dtype, device="cuda") for a in alone]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(threads), []

    def work(i):
        try:
            start.wait()
            for o in outs[i]:
                layer.forward(*batches[i], o, stream=0)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    workers = [threading.Thread(target=work, args=(i,)) for i in range(threads)]
    for w in workers:
        w.start()
    for w in workers:
        w.join()
    torch.cuda.synchronize()
    assert not errors
    for a, o in zip(alone, outs):
        assert (o == a).all(), f"{int((o != a).flatten(1).any(1).sum())} of {len(o)} calls"
