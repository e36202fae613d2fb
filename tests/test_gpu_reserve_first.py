"""sv_reserve_kv as the first call of a process, at sizes whose shared memory is
just below and just above what a kernel may take without asking."""

import os
import subprocess
import sys

import pytest

from speculative_decoding_verification_padding_gb300 import build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALL = """
import sys
import numpy as np
import torch
from oracle import edges
from speculative_decoding_verification_padding_gb300 import api
R, rows, chains = (int(x) for x in sys.argv[1:])
cu = np.arange(R + 1, dtype=np.int32) * rows
parent = None if chains else np.tile(np.arange(-1, rows - 1, dtype=np.int32), R)
ctx = (np.arange(R) * 7 % 40).astype(np.int32)
tables = np.full((R, 6), -1, np.int32)
used = 0
for i in range(R):
    n = -(-int(ctx[i]) // 16)
    tables[i, :n] = np.arange(used, used + n)
    used += n
free = np.arange(used, used + 4 * R, dtype=np.int32)
dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
out = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")
page = torch.empty(used + 4 * R, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
kv = api.PagedKV(page, page, dev(tables), dev(ctx))
N = int(cu[-1])
b = api.Batch(dev(cu), dev(parent), torch.zeros(N, dtype=torch.int32, device="cuda"), rows)
pool = api.BlockPool(dev(free), torch.tensor([len(free)], dtype=torch.int32, device="cuda"))
slots, positions, taken, status = out(N), out(N), out(R), torch.zeros(1, dtype=torch.int32, device="cuda")
api.sv_reserve_kv(kv, b, pool, slots, positions, taken, dev_status=status)
err, want = edges.reserve(cu, parent, ctx, tables, free, len(free), used + 4 * R, rows, N)
got = dict(tables=kv.block_tables, slots=slots, positions=positions, taken=taken)
assert err == status.item() == 0 and pool.free_count.item() == want["count"]
for k, t in got.items():
    assert np.array_equal(t.cpu().numpy(), want[k]), k
"""


@pytest.mark.parametrize("requests,rows,chains", [
    (2260, 1, 0), (2262, 1, 0), (2300, 1, 0),  # with parents, in one launch
    (2430, 15, 1), (2431, 15, 1), (2457, 15, 1), (2458, 15, 1)])  # more than 32768 rows, in two
def test_first_call_of_a_process(requests, rows, chains):
    build.build()
    r = subprocess.run([sys.executable, "-c", CALL, str(requests), str(rows), str(chains)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
