"""spmv_kv_append: what lands in the cache is the tokens bit for bit (or, in
an 8-bit cache, their nearest values), and nothing else changes."""
import numpy as np
import pytest
import torch

import load_balanced_csr_amd as lb
import kv_ref

pytestmark = pytest.mark.gpu
BITS = {4: torch.int32, 2: torch.int16, 1: torch.uint8}


def bits(t):
    return t.view(BITS[t.element_size()])


def pool(shape, dtype, heads_first, fill=3.0):
    n, P, H, D = shape
    if heads_first:
        return torch.full((n, H, P, D), fill, device="cuda").to(dtype).transpose(1, 2)
    return torch.full((n, P, H, D), fill, device="cuda").to(dtype)


def expect(cache, slots, rows):
    want = bits(cache).cpu().clone()
    P = cache.shape[1]
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < cache.shape[0] * P:
            want[s // P, s % P] = rows[t]
    return want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,D,P,heads_first", [
    (1, 1, 8, 1, False), (7, 3, 64, 16, True), (129, 8, 128, 24, False), (64, 5, 80, 7, True),
    (1000, 2, 256, 100, False), (33, 16, 96, 64, True)])
def test_append(dtype, T, H, D, P, heads_first):
    g = torch.Generator(device="cuda").manual_seed(T)
    n = T // P + 3
    k, v = pool((n, P, H, D), dtype, heads_first), pool((n, P, H, D), dtype, heads_first, 5.0)
    kn, vn = (torch.randn(T, H, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    kn[0, 0, :3] = torch.tensor([float("nan"), float("inf"), -0.0])
    slots = torch.randperm(n * P, device="cuda", generator=g)[:T].to(torch.int32)
    slots[T // 2::5] = -1
    slots[T // 3::7] = n * P
    wk, wv = expect(k, slots, bits(kn).cpu()), expect(v, slots, bits(vn).cpu())
    lb.KvCache(k, v).append(kn, vn, slots)
    assert torch.equal(bits(k).cpu(), wk) and torch.equal(bits(v).cpu(), wv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_append_of_strided_and_misaligned_rows(dtype):
    """Keys and values cut from one projection, heads outermost, and an odd start."""
    T, H, D, P = 37, 4, 64, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    both = torch.randn(T, 3, H, D, device="cuda", generator=g).to(dtype)
    flat = torch.randn(H * T * D + 1, device="cuda", generator=g).to(dtype)
    odd = flat[1:].view(H, T, D).transpose(0, 1)
    slots = torch.randperm(4 * P, device="cuda", generator=g)[:T].to(torch.int32)
    for kn, vn in ((both[:, 1], both[:, 2]), (odd, both[:, 0]), (both[:, 0], odd)):
        k, v = pool((4, P, H, D), dtype, False), pool((4, P, H, D), dtype, True)
        wk = expect(k, slots, bits(kn.contiguous()).cpu())
        wv = expect(v, slots, bits(vn.contiguous()).cpu())
        lb.KvCache(k, v).append(kn, vn, slots)
        assert torch.equal(bits(k).cpu(), wk) and torch.equal(bits(v).cpu(), wv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("scaled", [False, True])
def test_append_rounds_to_the_nearest_8_bit_value(dtype, scaled):
    T, H, D, P = 61, 3, 112, 16
    g = torch.Generator(device="cuda").manual_seed(11)
    spread = torch.exp(8 * torch.randn(T, H, D, device="cuda", generator=g))
    kn = (torch.randn(T, H, D, device="cuda", generator=g) * spread).clamp(-60000, 60000)
    kn = kn.to(dtype)
    kn[0, 0, :8] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 464.0, 448.0,
                                 2.0 ** -10, 3 * 2.0 ** -10])
    vn = torch.randn(T, H, D, device="cuda", generator=g).to(dtype)
    scale = 0.1 + torch.rand(2, H, device="cuda", generator=g) if scaled else None
    k, v = (pool((6, P, H, D), torch.float8_e4m3fn, hf) for hf in (False, True))
    slots = torch.randperm(6 * P, device="cuda", generator=g)[:T].to(torch.int32)
    want = []
    for i, (cache, new) in enumerate(((k, kn), (v, vn))):
        x = new.float().cpu().numpy()
        if scaled:
            x = x / scale[i].cpu().numpy()[None, :, None]
        want.append(expect(cache, slots, torch.from_numpy(kv_ref.to_e4m3(x))))
    cache = lb.KvCache(k, v, *(scale if scaled else (None, None)))
    cache.append(kn, vn, slots)
    for got, w in zip((k, v), want):
        got = bits(got).cpu()
        nan = (w & 0x7f) == 0x7f          # a NaN's sign is not kept by every rounding
        assert torch.equal(torch.where(nan, got & 0x7f, got), torch.where(nan, w & 0x7f, w))


def test_append_past_65536_tokens_and_of_none():
    P, H, D, T = 16, 1, 64, 70001
    k, v = pool((T // P + 1, P, H, D), torch.float16, False), pool((T // P + 1, P, H, D),
                                                                  torch.float16, False)
    kn = torch.randn(T, H, D, device="cuda").half()
    vn = torch.randn(T, H, D, device="cuda").half()
    slots = torch.randperm(T, device="cuda").to(torch.int32)
    cache = lb.KvCache(k, v)
    cache.append(kn[:0], vn[:0], slots[:0])
    cache.append(kn, vn, slots)
    flat = k.view(-1, H, D)[slots.long()], v.view(-1, H, D)[slots.long()]
    assert torch.equal(flat[0], kn) and torch.equal(flat[1], vn)


def test_append_on_another_stream():
    k, v = pool((40, 16, 2, 64), torch.bfloat16, False), pool((40, 16, 2, 64), torch.bfloat16, False)
    new = torch.randn(500, 2, 64, device="cuda").bfloat16()
    slots = torch.arange(500, device="cuda", dtype=torch.int32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lb.KvCache(k, v).append(new, new, slots, stream=s)
    s.synchronize()
    assert torch.equal(k.view(-1, 2, 64)[:500], new) and torch.equal(v.view(-1, 2, 64)[:500], new)


def test_append_refuses():
    k, v = (pool((4, 16, 2, 64), torch.bfloat16, False) for _ in range(2))
    cache, slots = lb.KvCache(k, v), torch.zeros(3, dtype=torch.int32, device="cuda")
    new = torch.zeros(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    for kn, vn, s, err in ((new[:, :1], new[:, :1], slots, ValueError),
                           (new, new[:2], slots, ValueError), (new, new, slots[:2], ValueError),
                           (new, new, slots.long(), TypeError),
                           (new.float(), new.float(), slots, lb.SpmvError),
                           (new, new.half(), slots, TypeError),
                           (k.view(-1, 2, 64)[:3], new, slots, lb.SpmvError)):
        with pytest.raises(err):
            cache.append(kn, vn, s)
