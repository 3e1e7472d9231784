"""The relative-position-bias attention on rows whose element offsets pass 32 bits, in every kernel: the
segments lie at the end of long tensors, of which nothing else is read or written."""
import pytest
import torch

from block_sparse_gqa_nsa_b200 import nsa
import relpos_bars as bars
import relpos_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("n_q,n_k,segs,lens_q,lens_k,heads,kv_heads,dim", [
    (3, 34_000_000, 2, [1, 2], [700, 40], 4, 1, 64),               # few queries
    (9_000_000, 9_000_000, 200_000, [64, 7, 0, 33], None, 4, 1, 64),   # short segments
    (68_000_000, 68_000_000, 850_000, [90, 130, 1], None, 1, 1, 32),   # 64 and 128 rows a CTA
    (34_000_000, 34_000_000, 2, [300, 500], None, 1, 1, 64),           # tensor-memory kernels
])
def test_offsets_past_32_bits(n_q, n_k, segs, lens_q, lens_k, heads, kv_heads, dim):
    same, lens_k = lens_k is None, lens_k or lens_q
    assert n_q * heads * dim > 2 ** 31 or n_k * kv_heads * dim > 2 ** 31
    g = torch.Generator().manual_seed(n_q)

    def table_of(lens, n):  # the first segments are empty and begin where the others do
        at = torch.tensor([n - sum(lens)] * (segs - len(lens) + 1) + lens).cumsum(0)
        at[:segs - len(lens) + 1] = n - sum(lens)
        at[segs - len(lens):] = n - sum(lens) + torch.tensor([0] + lens).cumsum(0)
        return at.int().cuda()

    off_q, off_k = table_of(lens_q, n_q), table_of(lens_k, n_k)

    def tail(n, lens, *shape, dtype=BF, make=torch.randn):
        x = torch.empty(n, *shape, dtype=dtype, device="cuda")
        t = x[n - sum(lens):]
        t.copy_(make(t.shape, generator=g))
        return x

    def places(shape, generator):
        return torch.randint(-9, 10, shape, generator=generator)

    pos_k = tail(n_k, lens_k, 1, dtype=torch.int32, make=places)
    pos_q = pos_k if same else tail(n_q, lens_q, 1, dtype=torch.int32, make=places)
    bucket_of = nsa.lsrm_relpos_log_buckets(8, 6).cuda()
    table = torch.randn(1, 8, heads, generator=g).to(BF).cuda()
    q, dout = (tail(n_q, lens_q, heads, dim) for _ in range(2))
    k, v = (tail(n_k, lens_k, kv_heads, dim) for _ in range(2))
    desc = nsa.make_relpos_desc(n_q, n_k, segs, heads, kv_heads, dim, 1, 8, 6)
    ws = nsa.relpos_workspace(desc)
    out, lse = torch.empty_like(q), torch.empty(n_q, heads, device="cuda")
    dq, dk, dv, dtable = (torch.empty_like(x) for x in (q, k, v, table))
    where = (off_q, off_k, pos_q, pos_k, bucket_of, table)
    nsa.lsrm_relpos_forward(desc, *where, q, k, v, out, lse, ws)
    nsa.lsrm_relpos_backward(desc, *where, q, k, v, out, lse, dout, dq, dk, dv, dtable, ws)
    assert nsa.lsrm_nsa_last_device_status(ws) == 0

    def near(x, lens):
        return x[x.shape[0] - sum(lens):]

    def near_off(lens):
        return torch.tensor([0] + lens).cumsum(0).int().cuda()

    args = (near_off(lens_q), near_off(lens_k), near(pos_q, lens_q), near(pos_k, lens_k), bucket_of, table,
            near(q, lens_q), near(k, lens_k), near(v, lens_k))
    want = ref.attention(*args)
    ref.check("out", near(out, lens_q), want["out"])
    ref.check("lse", near(lse, lens_q), want["lse"])
    grads = bars.gradients(*args, near(dout, lens_q))
    for n, x, lens in (("dq", dq, lens_q), ("dk", dk, lens_k), ("dv", dv, lens_k)):
        bars.check(n, near(x, lens), grads[n])
    bars.check("dtable", dtable, grads["dtable"])
