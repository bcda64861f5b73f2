"""Cases of the 8-bit head and of sampling run through both builds of the
library by tests/test_gpu_decode.py: the release build in the test process,
the bounds-checking debug build in a child process (FKL_LIBRARY). Run as a
script: python tests/decode_cases.py OUT.npz"""

import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def answer(fkl, h, head, head_scale, u, workspaces=None, outs=None, **settings):
    """Tokens answered by an 8-bit head: logits of the hidden states h, one draw for each row."""
    w, o = workspaces or {}, outs or {}
    logits = fkl.project(h, head, head_scale, out=o.get("logits"), workspace=w.get("project"))
    return (logits,) + fkl.sample(logits, u, token=o.get("token"), logprob=o.get("logprob"), workspace=w.get("sample"),
                                  **settings)


def make_head(fkl, torch, dev, N, K, V, seed, dtype=None):
    g = torch.Generator(device=dev).manual_seed(seed)
    h = torch.randn((N, K), generator=g, device=dev).to(dtype or torch.bfloat16)
    W = torch.randn((V, K), generator=g, device=dev).to(torch.bfloat16) * (3.0 / K ** 0.5)
    head, scale = fkl.quantize(W)
    return h, W, head, scale, torch.rand(N, generator=g, device=dev)


def run_all():
    import torch

    import output_projection_kl_amd as fkl
    dev = torch.device("cuda", 0)
    out = {}

    def keep(name, *ts):
        torch.cuda.synchronize()
        for i, t in enumerate(ts):
            out[f"{name}/{i}"] = t.float().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()

    g = torch.Generator(device=dev).manual_seed(5)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        x = torch.randn((9, 1003), generator=g, device=dev).to(dtype)
        keep(f"quantize {dtype}", *fkl.quantize(x[:, 2:900]))
    # every layout of the product, operands read in place and copied, ragged rows of the output
    for M, N, K in ((5, 70, 500), (9, 30001, 100), (60, 40001, 130), (38, 56217, 335), (117, 31149, 190),
                    (139, 19627, 283), (201, 32003, 287), (1030, 20003, 70), (505, 323, 7071), (3, 16, 9000)):
        a = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8, device=dev)
        b = torch.randint(-128, 128, (N, -(-K // 16) * 16), generator=g, dtype=torch.int8, device=dev)[:, :K]
        sa, sb = torch.rand(M, generator=g, device=dev), torch.rand(N, generator=g, device=dev) / K ** 0.5
        bias = torch.randn(N, generator=g, device=dev)
        store = torch.zeros((M, N + 5), device=dev, dtype=torch.bfloat16)
        print(f"[decode-cases] project {M} {N} {K}", flush=True)
        keep(f"project {M} {N} {K}", fkl.project(a, b, sb, a_scale=sa, bias=bias, out=store[:, 3:3 + N])[:, ::7])
    # every route of sampling
    for N, V, dtype in ((7, 100, torch.float32), (5, 1000, torch.bfloat16), (3, 1025, torch.float16),
                        (4, 20001, torch.float32), (40, 70001, torch.bfloat16), (2, 262137, torch.float16)):
        x = torch.randn((N, V + 9), generator=g, device=dev) * 2
        x[:, 5:25] += 9
        x[0] = float("-inf")
        x = x.to(dtype)[:, 3:3 + V]
        u = torch.rand(N, generator=g, device=dev)
        ids = torch.arange(V, dtype=torch.int32, device=dev).flip(0).repeat(N, 1)
        for s in (dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.95, temperature=1.8), dict(top_k=V // 2 + 1),
                  dict(min_p=0.1), dict(temperature=0.0), dict(top_p=0.9, min_p=0.01)):
            print(f"[decode-cases] sample {N} {V} {dtype} {s}", flush=True)
            keep(f"sample {N} {V} {dtype} {s}", *fkl.sample(x, u, ids=ids, **s))
    h, _, head, scale, u = make_head(fkl, torch, dev, 33, 136, 5000, 3)
    keep("answer", *answer(fkl, h, head, scale, u, top_k=50, top_p=0.95))
    return out


if __name__ == "__main__":
    np.savez(sys.argv[1], **run_all())
