"""The FFN-block operators called from two threads on two streams at once give, bit for bit, what they give alone."""
import threading

import pytest

pytestmark = pytest.mark.gpu

# every kernel of the linear: up to 8 rows, 9 to 32, K over a cluster, persistent tiles
LINEAR = [(1, 48, 1024), (8, 1024, 512), (16, 1024, 1024), (32, 520, 1040), (100, 512, 4096), (300, 1000, 1600),
          (700, 2048, 512)]


def _calls(seed):
    """A list of calls, each with inputs, weights and workspace of its own."""
    import torch
    from nvfp4_mixture_experts_expert_gb300 import api
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def linear(M, N, K):
        kb = -(-K // 128)
        a, w = normal(M, K).to(torch.float8_e4m3fn), normal(N, K).to(torch.float8_e4m3fn)
        sa, sw = torch.exp(normal(M, kb)), torch.exp(normal(-(-N // 128), kb))
        return lambda: (api.fp8_linear(a, sa, w, sw, out_dtype=torch.float32),)
    calls = [linear(*c) for c in LINEAR]
    for T, H, I, E, k in ((1, 1024, 512, 16, 4), (32, 512, 256, 24, 6), (3, 8192, 128, 2, 2), (2, 256, 4224, 2, 1)):
        w = api.quantize_moe_weights((normal(E, 2 * I, H) * 2 / H ** 0.5).bfloat16(),
                                     (normal(E, H, I) / I ** 0.5).bfloat16())
        layer, x, logits = api.MoEFewTokens(T, H, I, E, k), normal(T, H).bfloat16(), normal(T, E)
        calls.append(lambda layer=layer, x=x, logits=logits, w=w: (layer(x, logits, w),))
    x, res, w = normal(100, 1792).bfloat16(), normal(100, 1792).bfloat16(), normal(1792)
    calls.append(lambda: api.add_rms_norm_fp8(x, res, w))
    return calls


def test_two_threads_on_two_streams():
    import torch
    every = [_calls(seed) for seed in (1, 2)]
    want = [[[t.clone() for t in call()] for call in calls] for calls in every]
    torch.cuda.synchronize()
    failures, gate = [], threading.Barrier(2)

    def work(calls, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                for turn in range(20):
                    got = [call() for call in calls]
                    torch.cuda.current_stream().synchronize()
                    for i, (a, b) in enumerate(zip(got, want)):
                        if not all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b)):
                            failures.append((turn, i))
        except Exception as e:  # noqa: BLE001 -- reported by the main thread
            failures.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(every, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures[:5]


FIRST_CALLS = """
import sys, threading
sys.path[:0] = ["tests", "."]
import torch
import test_gpu_ffn_threads as T
calls = [T._calls(seed) for seed in (1, 1)]
torch.cuda.synchronize()
out, gate = [None, None], threading.Barrier(2)
def work(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        out[i] = []
        for call in calls[i]:
            gate.wait()
            out[i].append(call())
        torch.cuda.current_stream().synchronize()
threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
[t.start() for t in threads]
[t.join() for t in threads]
for a, b in zip(*out):
    for s, t in zip(a, b):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
print("equal")
"""


def test_first_calls_of_a_process_from_two_threads():
    """What a kernel's first launch works out (attributes, clusters that fit) is complete for the thread beside it."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(2):
        r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.split() == ["equal"], r.stdout + r.stderr
