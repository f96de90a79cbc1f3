"""The 8-bit operators in the debug build (-DPOETX_DEBUG: every TMA and bulk
copy checked before it is issued): no copy fails a check, and the results have
the release build's bits.  Each build runs in its own process, whose first
calls of all are captured into a graph, since a serving process may have no
other."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import os, sys
import numpy as np
import torch
sys.path.insert(0, os.environ["POETX_ROOT"])
from orthogonal_equivalence_b200 import build as pbuild
pbuild.build(debug=os.environ.get("POETX_DEBUG") == "1")
import orthogonal_equivalence_b200 as px

BF = torch.bfloat16
g = torch.Generator().manual_seed(0)
def rnd(*s): return torch.randn(*s, generator=g).cuda()
def codes(*s): return torch.randint(-128, 128, s, generator=g, dtype=torch.int8).cuda()

# (T, m, n): wide tiles of every width with and without a split of K, the pair
# kernel, rows that TMA cannot read or write whole
cases = []
for T, m, n in [(1, 512, 200), (20, 2048, 256), (50, 300, 129), (100, 1024, 640), (300, 512, 1000), (700, 9000, 512),
                (2500, 384, 1304), (2500, 200, 1301)]:
    cases.append((codes(T, m), rnd(T).abs(), codes(n, m), rnd(n).abs(), rnd(T, n).to(BF)))
x, r, gamma = rnd(300, 512).to(BF), rnd(300, 512).to(BF), rnd(512)
D, G = rnd(300, 512).to(BF), rnd(2, 256, 256).to(BF)
x2, D2, G2 = rnd(5000, 768).to(BF), rnd(5000, 768).to(BF), rnd(3, 256, 256).to(BF)

def run():
    out = []
    for xq, xs, Wq, ws, dz in cases:
        out += [px.matmul_int8(xq, xs, Wq, ws, BF), px.matmul_int8(xq, xs, Wq, ws, torch.float32),
                px.matmul_int8_grad(dz, Wq, ws), px.matmul_int8_grad(dz.float(), Wq, ws)]
    n = px.rmsnorm_quantize(x, gamma, r, y=True)
    out += [n.codes, n.scale, n.h, n.y, *px.rmsnorm_backward(D, n.h, gamma, n.rstd, r)]
    for a, d, w in ((x, D, G), (x2, D2, G2)):
        c = px.checkpoint_save(a)
        out += [c.codes, c.exps, px.checkpoint_load(c, BF), *px.block_backward(c, d, w),
                px.block_backward(c, d, w, need_o=False)[1]]
    return out

torch.cuda.synchronize()
px.lib()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
eager = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, eager)), "replayed and eager results differ"
out = {str(i): t.cpu().view(torch.uint8).numpy() for i, t in enumerate(t.contiguous() for t in eager)}
out["error"] = np.array([px.poetx_device_error()])
np.savez(sys.argv[1], **out)
"""


def _run(tmp_path, debug: bool):
    path = str(tmp_path / ("debug.npz" if debug else "release.npz"))
    env = dict(os.environ, POETX_ROOT=ROOT, POETX_DEBUG="1" if debug else "0")
    r = subprocess.run([sys.executable, "-c", SCRIPT, path], env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return dict(np.load(path))


def test_debug_build_checks_pass_and_match_release(tmp_path):
    rel = _run(tmp_path, False)
    dbg = _run(tmp_path, True)
    assert int(dbg["error"][0]) == 0, f"device error word {int(dbg['error'][0])} in the debug build"
    assert int(rel["error"][0]) == 0
    assert set(rel) == set(dbg)
    for k in rel:
        assert np.array_equal(rel[k], dbg[k]), k
