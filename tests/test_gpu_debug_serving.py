"""The chunk attention against the debug build (device-side index checks recorded in the error word): the
mixed and split batches of its tests leave no record, and a table entry outside the pool, which reads
zeros in either build, is reported."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUBSET = ["tests/test_gpu_chunk.py::test_mixed_batch", "tests/test_gpu_chunk.py::test_split_over_the_cache",
          "tests/test_gpu_chunk.py::test_few_rows_beside_many", "tests/test_gpu_serving_edges.py::test_deterministic",
          "tests/test_gpu_serving_edges.py::test_rows_without_keys_and_clamped_lengths"]

PROBE = r"""
import torch
import differential_attention_02_gb300 as da
P = 4
g = torch.Generator().manual_seed(5)
for fp8, d in ((False, 64), (False, 128), (True, 64), (True, 128)):
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    pages = [torch.randn(P, 2, 64, w, generator=g).to(dtype).cuda() for w in (d, d, 2 * d)]
    q = [torch.randn(20, 2, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = da.workspace(da.chunk_workspace_bytes(20, 1, 2, 1, 128, d, 2 * d))
    out = []
    for entry in (P + 3, 2):
        if entry == 2:
            for p in pages:
                p[2] = 0
        out.append(da.diffattn_chunk_paged(*q, *pages, i32([[0, entry]]), i32([0, 20]), i32([100]), 0.3, 0.2, L=128, ws=ws,
                                           scales=(1.0, 1.0, 1.0) if fp8 else None))
        print("CODE", da.read_error(ws))
    assert torch.equal(*out)
"""


@pytest.fixture(scope="module")
def env():
    from differential_attention_02_gb300 import build
    build.build()
    return {**os.environ, "DIFFATTN_LIBRARY": build.build(debug=True)}


def _python(args, env):
    r = subprocess.run([sys.executable, *args], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    return r.stdout


def test_batches_leave_no_record(env):
    assert " passed" in _python(["-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", *SUBSET], env)


def test_entries_outside_the_pool_are_reported(env):
    codes = [int(x.split()[1]) for x in _python(["-c", PROBE], env).splitlines() if x.startswith("CODE")]
    assert codes == [(0xC1 << 8) | 2, 0, (0xC3 << 8) | 2, 0] * 2
