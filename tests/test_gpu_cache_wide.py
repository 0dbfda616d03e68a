"""GPU: an 8-bit cache whose positions have more blocks of 32 than a CTA has threads (more than 8192 elements), up
to the most.  What is held and what is read back is compared exactly."""
from __future__ import annotations

import numpy as np
import pytest

from test_gpu_cache import TYPES, Case, dev, i32, same

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_61_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L,H,D,values", [(2, 128, 128, True), (1, 65, 128, True), (3, 9, 1008, False), (1, 64, 1024, True), (1, 1024, 48, True)])
def test_written_and_read(sv, dtype, L, H, D, values):
    """What a verify kept, a prompt behind it, and both read back, in pages of 5."""
    rng = np.random.default_rng(H + D)
    c = Case(L, 4, 5, H, D, rng, 5, values, held=6)
    count = 2 if values else 1
    k, n = np.array([3, 0, 5]), np.array([2, 0, 5])
    off = np.concatenate([[0], np.cumsum(k)])
    slots = np.array([2, 3, 0])
    x = [c.inputs(off[-1] + 3, dtype) for _ in range(count)]
    paths = [list(range(off[b] + b, off[b] + b + n[b] + 1)) for b in range(3)]
    for out in ("none", "new", "in place"):  # the same rows to the same places
        c.write(sv, x, paths, slots, off, out, rows="target", num_accepted=dev(n.astype(i32)))
    for r in c.refs:
        r.lengths = r.after
    x = [c.inputs(9, dtype) for _ in range(count)]
    c.write(sv, x, [list(range(9))], [1], [0, 9], "in place", rows="prompt")
    lengths = c.refs[0].after
    for r in c.refs:
        r.lengths = lengths
    off = np.concatenate([[0], np.cumsum(lengths)])
    R = off[-1] + 1
    out = tuple(None if i >= count else torch.full((L, R, H, D), 5.0, dtype=TYPES[dtype], device="cuda") for i in range(2))
    sv.spec_cache_read(*c.tensors, c.d_lengths, dev(off.astype(i32)), R, pages=c.d_pages, out=out)
    for g, r in zip(out, c.refs):
        want = torch.from_numpy(r.read(off, R, np.arange(4))).to(torch.float32).to(TYPES[dtype]).double().numpy()
        want[:, off[-1]:] = 5.0
        assert same(g.double().cpu().numpy(), want)
