"""Race check of the ragged, weight-gradient and 4-bit rings: every tile the library chooses gives the
same bits as the hand-off checking build (diag/libtbg_check.so, the same C ABI), where every stage
hand-off drains all copies and LDS reads first.  The log names the kernel each call took, so the
test also fails when a size no longer reaches the tile it stands for."""
import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHECK_LIB = os.path.join(ROOT, "tiled_bf16_gemm_amd", "diag", "libtbg_check.so")

# (call, sizes, the kernel the log must name); rows split evenly but for the last group
CASES = [
    ("grouped", dict(groups=2, M=5, N=90, K=200, layout="nk"), "rows 16x16"),
    ("grouped", dict(groups=40, M=600, N=500, K=400, layout="nk"), "ring 64x64"),
    ("grouped", dict(groups=40, M=600, N=500, K=400, layout="kn"), "ring 64x64"),
    ("grouped", dict(groups=8, M=2000, N=2048, K=4104, layout="nk"), "ring 128x128"),
    ("grouped", dict(groups=8, M=2000, N=2048, K=4104, layout="kn"), "ring 128x128"),
    ("grouped", dict(groups=8, M=5000, N=2048, K=4160, layout="nk"), "ring 256x256"),
    ("grouped", dict(groups=8, M=5000, N=2048, K=4160, layout="kn"), "ring 256x256"),
    ("wgrad", dict(groups=3, M=900, P=200, Q=150), "ring 64x64"),
    ("wgrad", dict(groups=64, M=2000, P=250, Q=200), "ring 128x128"),
    ("wgrad", dict(groups=2, M=5000, P=2048, Q=2060), "ring 256x256"),
    ("mx4", dict(M=3, N=300, K=2080), "rows 16x16"),
    ("mx4", dict(M=20, N=3000, K=2080), "ring 32x64, 4 stages"),
    ("mx4", dict(M=20, N=70000, K=2080), "ring 32x64, 2 stages"),
    ("mx4", dict(M=50, N=3000, K=2080), "ring 64x64, 4 stages"),
    ("mx4", dict(M=50, N=70000, K=1056), "ring 64x64, 2 stages"),
    ("mx4", dict(M=2000, N=2000, K=2080), "ring 128x128, 2 stages"),
    ("mx4", dict(M=4000, N=4000, K=4128), "ring 256x256, 2 stages"),
    # the sizes of the exact tests of the large tiles
    ("grouped", dict(groups=5, M=4009, N=3402, K=1276, layout="nk"), "ring 256x256"),
    ("grouped", dict(groups=5, M=4009, N=3402, K=1276, layout="kn"), "ring 256x256"),
    ("wgrad", dict(groups=5, M=6003, P=2003, Q=2058), "ring 256x256"),
    ("mx4", dict(M=5100, N=5003, K=2080), "ring 256x256, 2 stages"),
    ("mx4_grouped", dict(groups=5, M=6009, N=4603, K=2080), "ring 256x256, 2 stages"),
    ("mx4_grouped", dict(groups=4, M=8000, N=5003, K=2080), "ring 256x256, 2 stages"),
]


def _child():
    """Runs every case on both libraries; prints the log line markers and the verdicts."""
    sys.path.insert(0, ROOT)
    import torch
    import tiled_bf16_gemm_amd as tbg
    from tiled_bf16_gemm_amd import torch_ops as ops
    product, check = tbg._lib, ctypes.CDLL(CHECK_LIB)
    for n in ("tbg_gemm_grouped", "tbg_gemm_grouped_workspace_query", "tbg_gemm_grouped_wgrad",
              "tbg_gemm_grouped_wgrad_workspace_query", "tbg_mx4_gemm", "tbg_mx4_gemm_grouped", "tbg_mx4_quantize",
              "tbg_status_string", "tbg_last_error"):
        f, g = getattr(check, n), getattr(product, n)
        f.restype, f.argtypes = g.restype, g.argtypes
    gen = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    for i, (call, c, kernel) in enumerate(CASES):
        if call == "mx4":
            a, sa = ops.mx4_quantize(randn(c["M"], c["K"]))
            b, sb = ops.mx4_quantize(randn(c["N"], c["K"]))

            def run():
                return ops.mx4_gemm(a, sa, b, sb, "f32")
        elif call == "mx4_grouped":
            edges = [e * c["M"] // c["groups"] for e in range(c["groups"])] + [c["M"]]
            off = torch.tensor(edges, dtype=torch.int32, device="cuda")
            a, sa = ops.mx4_quantize(randn(c["M"], c["K"]))
            b, sb = ops.mx4_quantize(randn(c["groups"], c["N"], c["K"]))

            def run():
                return ops.mx4_gemm_grouped(a, sa, b, sb, off, "f32")
        else:
            edges = [e * c["M"] // c["groups"] for e in range(c["groups"])] + [c["M"] - 1]
            off = torch.tensor(edges, dtype=torch.int32, device="cuda")
            if call == "grouped":
                x = randn(c["M"], c["K"]).bfloat16()
                w = randn(c["groups"], *((c["N"], c["K"]) if c["layout"] == "nk" else (c["K"], c["N"]))).bfloat16()
                out = torch.zeros((c["M"], c["N"]), device="cuda")

                def run():
                    return ops.gemm_grouped(x, w, off, c["layout"], "f32", out=out)
            else:
                x, y = randn(c["M"], c["P"]).bfloat16(), randn(c["M"], c["Q"]).bfloat16()

                def run():
                    return ops.gemm_grouped_wgrad(x, y, off)
        for name, lib in (("lean", product), ("drained", check)):
            tbg._lib = lib
            print(f"case {i} {name}", file=sys.stderr, flush=True)
            r = run().clone()
            torch.cuda.synchronize()
            if name == "lean":
                lean = r
        tbg._lib = product
        print(f"verdict {i} {torch.equal(lean.view(torch.int32), r.view(torch.int32))}", flush=True)


@pytest.mark.gpu
def test_every_tile_matches_the_drained_build():
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True, timeout=110,
                       cwd=ROOT, env=dict(os.environ, TBG_LOG="1"))
    assert r.returncode == 0, r.stderr[-3000:]
    log = r.stderr.split("case ")[1:]
    assert len(log) == 2 * len(CASES)
    for i, (call, c, kernel) in enumerate(CASES):
        for part in log[2 * i:2 * i + 2]:
            assert kernel in part, (call, c, part)
        assert f"verdict {i} True" in r.stdout, (call, c)


if __name__ == "__main__":
    _child()
