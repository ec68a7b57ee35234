"""spmv_kv_attention against 64-bit sums over the visible tokens, in units of
error bounds that kv_ref.attend derives from the number formats."""
import math

import pytest
import torch

import load_balanced_csr_amd as lb
import kv_ref

pytestmark = pytest.mark.gpu

BF16, F16, F32, F8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


class Case:
    def __init__(self, lengths, Hq=8, H=2, D=128, P=16, dtype=BF16, heads_first=False, seed=0,
                 q_dtype=None, width=None, q_size=1.0):
        g = torch.Generator().manual_seed(seed)
        R = len(lengths)
        need = [kv_ref.pages_of(max(n, 0), P) for n in lengths]
        self.width = width or max(1, max(need, default=0)) + 1
        n_pages = sum(need) + 3
        perm = torch.randperm(n_pages, generator=g).to(torch.int32)
        self.table = torch.full((R, self.width), -1, dtype=torch.int32)
        at = 0
        used = torch.zeros(n_pages, P, dtype=torch.bool)
        for r, n in enumerate(need):
            self.table[r, :min(n, self.width)] = perm[at:at + n][:self.width]
            for j in range(n):
                used[perm[at + j].item(), :min(P, lengths[r] - j * P)] = True
            at += n
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        qd = q_dtype or (BF16 if dtype == F8 else dtype)
        self.q = (torch.randn(R, Hq, D, generator=g) * q_size).to(qd)
        shape = (n_pages, P, H, D)
        self.k = (torch.randn(shape, generator=g) * (8 if dtype == F8 else 1)).to(dtype)
        self.v = (torch.randn(shape, generator=g) * (8 if dtype == F8 else 1)).to(dtype)
        self.scales = None
        if dtype == F8:
            self.scales = 0.05 + 0.1 * torch.rand(2, H, generator=g)
        # what no request holds is poison
        for t in (self.k, self.v):
            if dtype == F8:
                t.view(torch.uint8)[~used] = 0x7f
            else:
                t[~used] = float("nan")
        self.heads_first = heads_first
        self.scale = D ** -0.5

    def cache(self):
        def put(t):
            if not self.heads_first:
                return t.cuda()
            return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        self.gk, self.gv = put(self.k), put(self.v)
        s = (None, None) if self.scales is None else tuple(self.scales.cuda())
        return lb.KvCache(self.gk, self.gv, *s)

    def ref(self, **kw):
        s = {} if self.scales is None else dict(k_scale=self.scales[0], v_scale=self.scales[1])
        return kv_ref.attend(self.q, self.k, self.v, self.table, self.lengths, self.scale, **kw,
                             **s)

    def check(self, cache=None, **kw):
        cache = cache or self.cache()
        q, table, lengths = self.q.cuda(), self.table.cuda(), self.lengths.cuda()
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        out = torch.full_like(q, 7.0)
        cache.attend(q, table, lengths, out, lse=lse, **kw)
        torch.cuda.synchronize()
        ref, rlse, tol, ltol = self.ref(**kw)
        assert kv_ref.worst(out, ref, tol) <= 1.0, kv_ref.worst(out, ref, tol)
        assert kv_ref.worst(lse, rlse, ltol) <= 1.0, kv_ref.worst(lse, rlse, ltol)
        return out, lse


@pytest.mark.parametrize("dtype", [BF16, F16, F32, F8])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256,
                               257, 513])
def test_lengths_about_every_tile_edge(dtype, n):
    Case([n, 5, n], dtype=dtype, seed=n).check()


@pytest.mark.parametrize("dtype", [BF16, F16, F32, F8])
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 256])
def test_head_sizes(dtype, D):
    Case([70, 1, 200, 0, 33], D=D, Hq=6, H=3, dtype=dtype, seed=D).check()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [8, 24, 40, 72, 88, 120, 136, 200, 248])
def test_head_sizes_that_are_odd_multiples_of_8(dtype, D):
    Case([70, 1, 40], D=D, Hq=3, H=1, dtype=dtype, seed=D).check()


@pytest.mark.parametrize("D", [4, 12, 20, 36, 60, 68, 100, 132, 252])
def test_head_sizes_that_are_odd_multiples_of_4(D):
    Case([70, 1, 40], D=D, Hq=3, H=1, dtype=F32, seed=D).check()


@pytest.mark.parametrize("dtype", [BF16, F32, F8])
@pytest.mark.parametrize("H,G", [(1, 1), (4, 1), (3, 2), (2, 3), (2, 5), (1, 7), (2, 8), (1, 15),
                                 (2, 16), (1, 17), (1, 24), (2, 32), (1, 33), (1, 48), (1, 71)])
def test_groups_of_query_heads(dtype, H, G):
    Case([90, 300, 7], Hq=H * G, H=H, D=64, dtype=dtype, seed=H * 100 + G).check()


@pytest.mark.parametrize("dtype", [BF16, F32, F8])
@pytest.mark.parametrize("P", [1, 2, 3, 7, 8, 16, 24, 32, 64, 100, 128, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_page_sizes_and_layouts(dtype, P, heads_first):
    Case([129, 31, 300], D=64, P=P, dtype=dtype, heads_first=heads_first, seed=P).check()


@pytest.mark.parametrize("dtype", [BF16, F16, F32, F8])
def test_an_8_bit_or_other_cache_with_either_query_type(dtype):
    for qd in (BF16, F16) if dtype == F8 else (dtype,):
        Case([200, 64, 3], dtype=dtype, q_dtype=qd).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 4), (31, 33), (64, 0), (100, 17),
                                          (200, 200), (1000, 4), (128, 1), (97, 128)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_windows_and_sinks(dtype, window, sinks):
    Case([0, 1, 30, 64, 100, 101, 333, 700], D=64, P=24, dtype=dtype,
         seed=window).check(window=window, sinks=sinks)


def test_window_keeps_poison_outside_out():
    """Tokens that the window hides hold NaN: none of it may show."""
    c = Case([400, 129], D=64, seed=3)
    for r, n in enumerate((400, 129)):
        for t in range(2, n - 50):
            p, i = c.table[r, t // 16].item(), t % 16
            c.k[p, i] = float("nan")
            c.v[p, i] = float("inf")
    out, _ = c.check(window=50, sinks=2)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype,n", [(BF16, 40000), (F32, 9001), (F8, 20011)])
def test_long_rows_are_split_and_joined(dtype, n):
    Case([n, 3, n // 3], Hq=4, H=1, D=128, P=64, dtype=dtype).check()


@pytest.mark.parametrize("dtype,D,G", [(BF16, 256, 24), (F8, 256, 17), (F16, 128, 32), (F32, 256, 5),
                                       (BF16, 192, 40), (F8, 128, 3), (F32, 80, 20)])
def test_wide_heads_and_groups_joined_either_way(dtype, D, G):
    """Few rows (their parts joined by a second launch), then more than 64 with a long one
    among them (joined by the workgroups, in two levels), in whole pages and odd ones."""
    for P in (64, 20):
        Case([6000, 3, 40], Hq=G, H=1, D=D, P=P, dtype=dtype, seed=G).check()
        Case([9000] + [5] * 70 + [0], Hq=G, H=1, D=D, P=P, dtype=dtype, seed=G + 1).check()


def test_long_rows_beside_many_short_ones():
    Case([1 + 13 * (r % 9) for r in range(150)] + [9000] + [0, 1] * 20, Hq=8, H=2, D=64,
         seed=7).check()


def test_more_rows_than_one_scan_chunk():
    Case([r % 5 for r in range(1300)], Hq=2, H=2, D=64, P=2).check()


def test_every_row_empty():
    out, lse = Case([0, 0, 0]).check()
    assert (out == 0).all() and (lse == -math.inf).all()


def test_lengths_out_of_range():
    """Below 0 counts as 0; past the table's width, as that."""
    c = Case([40, 33, 64], width=3, D=64)
    c.lengths = torch.tensor([-7, 2 ** 31 - 1, 64], dtype=torch.int32)
    c.table[1] = torch.tensor([c.table[1, 0], c.table[1, 1], c.table[1, 0]])
    c.k = torch.nan_to_num(c.k, nan=0.5)
    c.v = torch.nan_to_num(c.v, nan=0.5)
    c.check()


def test_pages_outside_the_cache_are_not_visible():
    c = Case([200, 100, 16], D=64, seed=5)
    c.table[0, 3] = -1
    c.table[0, 7] = 10 ** 6
    c.table[1, 0] = -(2 ** 31)
    c.table[2, 0] = 2 ** 31 - 1                      # the whole row
    out, lse = c.check()
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()


def test_scores_far_from_zero():
    """Scores of some thousands, the largest at the start, in the middle, at the end."""
    for place in (0, 150, 299):
        c = Case([300, 300], D=64, dtype=F32, q_size=30.0)
        c.k[c.table[0, place // 16].item(), place % 16] *= 20
        c.check()


def test_values_of_the_types_ends():
    """The type's lowest value as a key (a row of it alone and beside others), infinities and
    NaN in visible places: as the formula has them."""
    c = Case([40, 40, 40, 1], D=64, Hq=2, H=1, dtype=F32)
    low = torch.finfo(F32).min
    c.q[0] = 0.0
    c.k[c.table[0, 0].item(), 3] = 1e30
    c.q[1, :, 0] = c.q[1, :, 0].abs() + 1.0
    c.k[c.table[1, 1].item(), 5, :, 0] = low / 1e30        # a score that exp() sends to 0
    c.v[c.table[2, 1].item(), 2, 0, 7] = float("inf")
    out, lse = c.check()
    assert out[2, 0, 7] == math.inf and torch.isfinite(lse[:3]).all()
    c.k[c.table[2, 0].item(), 1] = float("nan")
    c.k[c.table[3, 0].item(), 0, 0, 0] = float("inf")
    c.q[3, 0, 0], c.q[3, 1, 0] = 1.0, -1.0
    got = c.cache().attend(c.q.cuda(), c.table.cuda(), c.lengths.cuda()).cpu()
    assert torch.isnan(got[2]).all() and torch.isnan(got[3, 0]).all()
    # every score -inf: as if no token were visible
    assert (got[3, 1] == 0).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: pages at its end are read where they are."""
    P, H, D, n_pages = 16, 8, 128, 300_000
    k = torch.empty(n_pages, P, H, D, dtype=BF16, device="cuda")
    v = torch.empty(n_pages, P, H, D, dtype=BF16, device="cuda")
    c = Case([100, 37], Hq=16, H=H, D=D)
    far = torch.tensor([n_pages - 1, 0, 262_144, n_pages - 2, 131_072, 262_143, 7, 299_000, 262_145,
                        199_999, 65_536, 5, 77])
    assert k.numel() > 2 ** 32 and c.k.shape[0] <= far.numel()
    far = far[:c.k.shape[0]]
    k[far.cuda()], v[far.cuda()] = c.k.cuda(), c.v.cuda()
    want = c.ref()
    table = torch.where(c.table >= 0, far[c.table.clamp(min=0).long()], -1).to(torch.int32)
    out = lb.KvCache(k, v).attend(c.q.cuda(), table.cuda(), c.lengths.cuda())
    assert kv_ref.worst(out, want[0], want[2]) <= 1.0


def test_tokens_far_apart_within_a_page():
    """Tokens outermost in memory, 2^24 elements from one to the next."""
    c = Case([50, 33, 16], Hq=4, H=1, D=64)
    n_pages = 2 ** 18
    want = c.ref()
    caches = []
    for t in (c.k, c.v):
        far = torch.empty(16, n_pages, 1, 64, dtype=BF16, device="cuda").transpose(0, 1)
        far[:t.shape[0]] = t.cuda()
        caches.append(far)
    assert caches[0].stride(1) == 2 ** 24
    out = lb.KvCache(*caches).attend(c.q.cuda(), c.table.cuda(), c.lengths.cuda())
    assert kv_ref.worst(out, want[0], want[2]) <= 1.0


def test_a_table_as_wide_as_tables_get():
    """2^31 - 2048 tokens of room in each of 20 rows: shares are dealt in several steps."""
    c = Case([0, 1, 5000, 63, 64, 65, 300, 2, 1100, 1024] * 2, Hq=4, H=2, D=64, P=1024)
    want = c.ref()
    wide = torch.full((20, 2 ** 21 - 2), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.width] = c.table.cuda()
    out = c.cache().attend(c.q.cuda(), wide, c.lengths.cuda())
    assert kv_ref.worst(out, want[0], want[2]) <= 1.0


def test_strided_queries_outputs_and_tables():
    c = Case([100, 3, 260, 64], Hq=6, H=3, D=80, dtype=F16)
    want = c.ref()
    cache = c.cache()
    R, Hq, D = c.q.shape
    qkv = torch.zeros(R, 12, D, dtype=F16, device="cuda")
    qkv[:, 2:8] = c.q.cuda()
    odd = torch.zeros(R * Hq * D + 1, dtype=F16, device="cuda")[1:].view(R, Hq, D)
    odd.copy_(c.q)
    turned = c.q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    wide = torch.full((R, c.width + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + c.width] = c.table.cuda()
    table = wide[:, 2:2 + c.width]
    for q in (qkv[:, 2:8], odd, turned):
        buf = torch.full((Hq, R, D + 3), 9.0, dtype=F16, device="cuda")
        for out in (buf[:, :, :D].transpose(0, 1), torch.empty(R, Hq, D, dtype=F16, device="cuda")):
            cache.attend(q, table, c.lengths.cuda(), out)
            assert kv_ref.worst(out, want[0], want[2]) <= 1.0
        assert (buf[:, :, D:] == 9.0).all()


def test_results_are_the_same_bits_every_time_and_on_another_stream():
    c = Case([5000, 17, 0, 2500, 1] + [400] * 30, Hq=16, H=2, D=128, seed=2)
    cache = c.cache()
    q, table, lengths = c.q.cuda(), c.table.cuda(), c.lengths.cuda()
    first = cache.attend(q, table, lengths).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for i in range(30):
        out = cache.attend(q, table, lengths, stream=s if i % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(out, first), i


def test_calls_on_two_streams_at_once():
    """One cache, calls that split rows on two streams with nothing between them: each
    stream has a workspace of its own."""
    c = Case([7000, 300, 5], Hq=8, H=2, D=128, seed=6)
    cache = c.cache()
    q, table, lengths = c.q.cuda(), c.table.cuda(), c.lengths.cuda()
    want = cache.attend(q, table, lengths)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, out in zip(streams, outs):
            cache.attend(q, table, lengths, out[i], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for out in outs for o in out)


def test_a_workspace_serves_calls_of_other_shapes():
    """One workspace, calls that split long rows and calls that do not, in turn."""
    cases = [Case([6000, 100], Hq=8, H=2, D=128), Case([3] * 40, Hq=8, H=2, D=128, seed=1),
             Case([1, 0, 9000], Hq=8, H=2, D=128, seed=2)]
    need = max(c.cache().workspace_size(8) for c in cases)
    ws = torch.full((max(need, 16),), 0xa5, dtype=torch.uint8, device="cuda")
    ws[:lb.kv.KV_WORKSPACE_ZEROED] = 0
    wants = [c.ref() for c in cases]
    for turn in range(3):
        for c, w in zip(cases, wants):
            out = c.cache().attend(c.q.cuda(), c.table.cuda(), c.lengths.cuda(), workspace=ws)
            assert kv_ref.worst(out, w[0], w[2]) <= 1.0


def test_graph_replays_match_the_eager_calls():
    """Captured once, replayed as the lengths grow."""
    c = Case([3000, 40, 0, 700], Hq=8, H=2, D=128, seed=4)
    cache = c.cache()
    q, table = c.q.cuda(), c.table.cuda()
    lengths = torch.tensor([2000, 30, 0, 100], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    step = torch.tensor([50, 1, 0, 30], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cache.attend(q, table, lengths, out, stream=s)     # the stream's workspace, before capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cache.attend(q, table, lengths, out)
    for i in range(10):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, cache.attend(q, table, lengths)), i
        lengths += step


def test_the_formula_s_join():
    """Attention over two halves of a row, joined by their lse, is that over the row."""
    c = Case([600], Hq=4, H=2, D=64, dtype=F32)
    cache = c.cache()
    q, table, n = c.q.cuda(), c.table.cuda(), c.lengths.cuda()
    parts = []
    for t, m in ((table[:, :16], 256), (table[:, 16:], 344)):
        lse = torch.empty(1, 4, device="cuda")
        parts.append((cache.attend(q, t.contiguous(), torch.full_like(n, m), lse=lse), lse))
    w = torch.softmax(torch.stack([l for _, l in parts]), 0)
    joined = sum(w[i][..., None] * parts[i][0] for i in range(2))
    ref, _, tol, _ = c.ref()
    assert kv_ref.worst(joined, ref, 4 * tol) <= 1.0


def test_attention_refuses():
    c = Case([20, 3], D=64)
    cache = c.cache()
    q, table, n = c.q.cuda(), c.table.cuda(), c.lengths.cuda()
    need = cache.workspace_size(8)
    bad = [(dict(q=q[:, :, :32]), ValueError), (dict(q=q.float()), lb.SpmvError),
           (dict(q=q[:, :7]), lb.SpmvError), (dict(out=q), lb.SpmvError),
           (dict(out=torch.empty_like(q[:1])), ValueError), (dict(table=table[:1]), ValueError),
           (dict(table=table.long()), TypeError), (dict(lengths=n[:1]), ValueError),
           (dict(lengths=n.long()), TypeError), (dict(window=-1), lb.SpmvError),
           (dict(sinks=-1), lb.SpmvError), (dict(scale=math.nan), lb.SpmvError),
           (dict(lse=torch.empty(2, 8, device="cuda", dtype=F16)), TypeError),
           (dict(lse=torch.empty(2, 7, device="cuda")), ValueError), (dict(q=c.q), ValueError)]
    if need:
        bad.append((dict(workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda")),
                    lb.SpmvError))
    for kw, err in bad:
        a = dict(q=q, table=table, lengths=n)
        a.update(kw)
        with pytest.raises(err):
            cache.attend(**a)
