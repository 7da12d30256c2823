"""The serving operators on the GPU against the fp64 oracle on the same inputs.

Tolerances, derived from the arithmetic (u = eps / 2 of the output's type):
  rotation  a pair's angle is off by at most 1.5e-6 rad (the fp64 product at
            positions up to 2^31, its fraction and sincospi in fp32), two
            products and a sum in fp32 add 2^-22: |dy| <= u |y| +
            (1.5e-6 + 2^-22)(|a| + |b|), plus half the least subnormal.
  scores    128 products of 16-bit values summed in fp32, at most 2^-23 of the
            magnitudes lost per addition: ds = 128 2^-23 S, S = max_j sum_d
            |q_d k_jd| / sqrt(d); the shifted exponent and 2^x add 2^-20 plus
            2^-23 of the score itself.  e = ds + 2^-20 + 2^-23 S.
  sums      n keys in steps of 16 and at most 300 joins: (n / 16 + 300) 2^-23.
  output    P is rounded to 16 bits (u_t) before the product with V; with A =
            the softmax mean of |v|: |do| <= u |o| + (u_t + 2 e + sums) A;
            fp16 probabilities below 2^-14 (of sums that are at least 2^7) lose
            at most 2^-25: n 2^-32 max|v|.
  lse       |d lse| <= e + sums + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

import score_keys_pooled_b200 as s2o
from score_keys_pooled_b200 import synth
from oracle import serve_oracle as SO
from tests import serve_ways as ways

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BAD_CACHE = 8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    s2o.lib()


def f64(t):
    return t.double().cpu().numpy()


def half_step(t):
    return torch.finfo(t).eps / 2


def assert_rotated(got, want, mag, t, what=""):
    tol = half_step(t) * np.abs(want) + (1.5e-6 + 2.0 ** -22) * mag + torch.finfo(t).smallest_normal * half_step(t)
    bad = np.abs(f64(got) - want) > tol
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist())


# --- rotation -----------------------------------------------------------------------------------------


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("rot,sections,adjacent", [
    (128, None, False), (128, None, True), (128, (16, 24, 24), False), (64, (10, 22), True), (16, None, False),
    (32, (0, 16), False), (96, (1, 46, 1), True), (0, None, False)])
def test_rotary_matches_the_oracle(t, rot, sections, adjacent):
    t = TYPES[t]
    r = s2o.make_rotary(rot, theta=500000.0, sections=sections, interleaved=adjacent)
    g = torch.Generator(device="cuda").manual_seed(rot)
    for B, N, Hq, Hkv in ((1, 1, 1, 1), (2, 37, 5, 3), (3, 9, 0, 2), (1, 200, 4, 0)):
        qkv = torch.randn(B, N, Hq + 2 * Hkv, 128, generator=g, device="cuda").to(t)
        q = qkv[:, :, :Hq] if Hq else None
        k = qkv[:, :, Hq:Hq + Hkv] if Hkv else None
        pos = torch.randint(0, 100000, (r.naxes, B, N), generator=g, device="cuda", dtype=torch.int32)
        for inverse in (False, True):
            out = s2o.rotary(r, q, k, pos, inverse=inverse)
            assert s2o.last_launch_count() == 1
            for x, y in zip((q, k), out):
                if x is None:
                    assert y is None
                    continue
                assert (y.transpose(1, 2) if not inverse else y).is_contiguous()
                for b in range(B):
                    want, mag = SO.rotate(f64(x[b]), pos[:, b].cpu().numpy(), rot, r.axis, r.inv_freq, adjacent, inverse)
                    assert_rotated(y[b], want, mag, t, (B, N, inverse))
    assert s2o.last_device_error() == 0


def test_rotary_at_far_and_negative_positions():
    r = s2o.make_rotary(128, theta=1e6)
    pos = torch.tensor([0, 1, 131071, 1 << 24, (1 << 31) - 1, -5, -(1 << 31)], dtype=torch.int64).to(torch.int32)
    x = torch.randn(1, 7, 2, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    y, _ = s2o.rotary(r, x, None, pos.view(1, 1, 7).cuda())
    want, mag = SO.rotate(f64(x[0]), pos.numpy()[None], 128, r.axis, r.inv_freq)
    assert_rotated(y[0], want, mag, torch.bfloat16)


def test_rotary_in_place_into_views_and_between():
    """In place; a head-major output inside a larger buffer whose rest stays; the
    inverse of the rotation gives the input back to within two roundings."""
    r = s2o.make_rotary(64, sections=(8, 24))
    x = torch.randn(2, 33, 3, 128, device="cuda").half()
    pos = torch.arange(2 * 2 * 33, device="cuda", dtype=torch.int32).view(2, 2, 33)
    want, _ = s2o.rotary(r, x, None, pos)
    y = x.clone()
    s2o.rotary(r, None, y, pos, k_out=y)
    assert torch.equal(y, want)
    big = torch.full((2, 5, 40, 128), 7.0, device="cuda", dtype=torch.float16)
    s2o.rotary(r, x, None, pos, q_out=big[:, 1:4, 2:35].transpose(1, 2))
    assert torch.equal(big[:, 1:4, 2:35].transpose(1, 2), want)
    big[:, 1:4, 2:35] = 7.0
    assert bool((big == 7.0).all())
    back, _ = s2o.rotary(r, want, None, pos, inverse=True)
    mag = x.abs() + x.abs()[..., list(range(32, 64)) + list(range(32)) + list(range(64, 128))]
    assert bool(((back - x).double().abs() <= 2 * half_step(torch.float16) * 1.5 * mag.double() + 1e-6).all())


def test_rotary_in_one_buffer():
    """Queries and keys side by side in one buffer, in place and from one into
    another, token-major and head-major: views that lie within one another's reach
    and share no row."""
    r = s2o.make_rotary(128)
    B, N, Hq, Hkv = 2, 19, 6, 2
    pos = torch.arange(B * N, device="cuda", dtype=torch.int32).view(1, B, N)
    packed = torch.randn(B, N, Hq + 2 * Hkv, 128, device="cuda").bfloat16()
    q, k, v = packed[:, :, :Hq], packed[:, :, Hq:Hq + Hkv], packed[:, :, Hq + Hkv:].clone()
    wq, wk = (x.clone() for x in s2o.rotary(r, q, k, pos))
    heads = torch.empty(B, Hq + Hkv, N, 128, device="cuda", dtype=torch.bfloat16)
    hq, hk = heads[:, :Hq].transpose(1, 2), heads[:, Hq:].transpose(1, 2)
    s2o.rotary(r, q, k, pos, q_out=hq, k_out=hk)
    assert torch.equal(hq, wq) and torch.equal(hk, wk)
    s2o.rotary(r, q, k, pos, q_out=q, k_out=k)
    assert torch.equal(q, wq) and torch.equal(k, wk) and torch.equal(packed[:, :, Hq + Hkv:], v)
    s2o.rotary(r, hq[:, :, 3:], hq[:, :, :3], pos, q_out=hq[:, :, 3:], k_out=hq[:, :, :3], inverse=True)
    assert s2o.last_device_error() == 0
    for bad in (dict(q_out=hq[:, :, :3], k_out=hq[:, :, 2:4]), dict(q_out=hq[:, :, 1:4], k_out=hk)):
        with pytest.raises(s2o.S2OError) as e:
            s2o.rotary(r, hq[:, :, :3], hk, pos, **bad)
        assert e.value.code == 1 and s2o.last_launch_count() == 0


def test_dimensions_of_one_may_have_any_stride():
    """One batch, one token, one head: torch leaves odd strides there."""
    r = s2o.make_rotary(128)
    pos = torch.full((1, 1, 1), 77, device="cuda", dtype=torch.int32)
    x = torch.randn(1, 1, 1, 128, device="cuda").bfloat16()
    want, _ = s2o.rotary(r, x, None, pos)
    odd = x.as_strided((1, 1, 1, 128), (1, 3, 5, 1))
    out = torch.empty_like(x).as_strided((1, 1, 1, 128), (7, 1, 1, 1))
    s2o.rotary(r, odd, None, pos, q_out=out)
    assert torch.equal(out, want)
    y = torch.randn(5, 128, 1, device="cuda").bfloat16().transpose(1, 2)  # [5, 1, 128], head stride 1
    assert y.stride(1) == 1
    pos = torch.arange(5, device="cuda", dtype=torch.int32).view(1, 1, 5)
    want, _ = s2o.rotary(r, y.contiguous()[None], None, pos)
    got, _ = s2o.rotary(r, y[None], None, pos)
    assert torch.equal(got, want)
    b = Batch([5], [9], Hq=1, Hkv=1)
    kc, vc = b.k.cuda(), b.v.cuda()
    s2o.cache_append(b.cfg, None, y, y, kc, vc, b.table.cuda(), b.q_start.cuda(), b.kv_len.cuda())
    assert s2o.last_device_error() == 0
    assert torch.equal(kc[b.table[0, 0].long(), 0, 4:9], y[:, 0]) and torch.equal(vc[b.table[0, 0].long(), 0, 4:9], y[:, 0])


# --- append -------------------------------------------------------------------------------------------


class Batch:
    """Sequences of a paged cache on the GPU; everything a call may not read is
    NaN: pages of nobody, rows behind the lengths, table entries behind the pages."""

    def __init__(self, new, length, P=0, page=16, Hq=8, Hkv=2, t=torch.bfloat16, seed=0, extra_rows=0, max_q=None,
                 max_pages=None, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.want = None
        self.new, self.len, self.P, self.page, self.t = list(new), list(length), P, page, t
        nseq, own = len(new), sum(new)
        self.own, self.Tq = own, own + extra_rows
        max_pages = max_pages or max(1, max(-(-n // page) for n in length)) + 1
        pre, used = -(-P // page), [-(-n // page) for n in length]
        num_pages = pre + sum(used) + 2
        ids = torch.randperm(num_pages, generator=g).int()
        self.prefix_pages = ids[:pre].clone()
        self.table = torch.full((nseq, max_pages), -1, dtype=torch.int32)
        at = pre
        for s, n in enumerate(used):
            self.table[s, :n] = ids[at:at + n]
            at += n
        self.q_start = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        self.kv_len = torch.tensor(length, dtype=torch.int32)
        self.k, self.v = (torch.full((num_pages, Hkv, page, 128), float("nan"), dtype=t) for _ in range(2))
        self.fill(self.prefix_pages, P, g, scale)
        for s in range(nseq):
            self.fill(self.table[s], length[s], g, scale)
        self.q = (scale * torch.randn(self.Tq, Hq, 128, generator=g)).to(t)
        self.cfg = s2o.make_cache(Hq, Hkv, page, num_pages, nseq, max_pages, self.Tq,
                                  max_q=max_q or max(1, max(new)), prefix_len=P,
                                  dtype=s2o.FP16 if t is torch.float16 else s2o.BF16)

    def fill(self, pages, n, g, scale):
        for i in range(-(-n // self.page)):
            m = min(self.page, n - i * self.page)
            for c in (self.k, self.v):
                c[pages[i], :, :m] = (scale * torch.randn(c.shape[1], m, 128, generator=g)).to(self.t)

    def dev(self):
        return [x.cuda() for x in (self.q, self.k, self.v, self.table, self.q_start, self.kv_len, self.prefix_pages)]

    def check(self, O, lse, what=""):
        """Against the oracle, rows behind the last sequence left out."""
        if self.want is None:
            self.want = SO.attend(f64(self.q), f64(self.k), f64(self.v), self.table.numpy(), self.q_start.numpy(),
                                  self.kv_len.numpy(), self.prefix_pages.numpy(), self.P)
        want, wl, A, S, n = self.want
        m = self.own
        want, wl, A, S, n = want[:m], wl[:m], A[:m], S[:m], n[:m]
        u, ut = half_step(O.dtype), half_step(self.t)
        e = 128 * 2.0 ** -23 * S + 2.0 ** -20 + 2.0 ** -23 * S
        sums = (n[:, None] / 16 + 300) * 2.0 ** -23
        tol = u * np.abs(want) + (ut + 2 * e + sums)[..., None] * A
        if self.t is torch.float16:
            vmax = float(np.nanmax(np.abs(f64(self.v))))
            tol += (n[:, None, None] * 2.0 ** -32 * vmax) + 2.0 ** -25
        bad = ~(np.abs(f64(O[:m]) - want) <= tol)
        assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                               f64(O[:m])[bad][:3].tolist(), want[bad][:3].tolist())
        if lse is not None:
            ok = np.abs(f64(lse[:m]) - wl) <= e + sums + 2.0 ** -22 * np.abs(wl)
            assert ok.all(), (what, np.argwhere(~ok)[:3].tolist())


def attend(b, **kw):
    q, k, v, table, qs, kl, pre = b.dev()
    O, lse = s2o.attention_paged(b.cfg, q, k, v, table, qs, kl, prefix_pages=pre, **kw)
    assert s2o.last_device_error() == 0
    return O, lse


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("new,length,P,page,axes,adjacent", [
    ([1], [1], 0, 16, 1, False),
    ([1] * 5, [1, 16, 17, 64, 100], 33, 16, 1, False),
    ([7, 0, 1, 40, 0], [7, 5, 130, 77, 0], 0, 32, 3, True),
    ([130, 3], [200, 3], 1000, 128, 2, False),
])
def test_append_writes_the_rows_it_should_and_no_others(t, new, length, P, page, axes, adjacent):
    t = TYPES[t]
    b = Batch(new, length, P, page, t=t, extra_rows=3, seed=len(new))
    sections = {1: None, 2: (30, 34), 3: (16, 24, 24)}[axes]
    r = s2o.make_rotary(128, theta=500000.0, sections=sections, interleaved=adjacent)
    g = torch.Generator().manual_seed(9)
    qkv = torch.randn(b.Tq, 12, 128, generator=g).to(t)  # packed projection: strided views
    k0, v0 = b.k.clone(), b.v.clone()
    pos = torch.randint(0, 5000, (axes, b.Tq), generator=g, dtype=torch.int32) if axes > 1 else None
    d = qkv.cuda()
    kc, vc = k0.cuda(), v0.cuda()
    q_out = torch.full((b.Tq, 8, 128), 3.0, device="cuda", dtype=t)
    got = s2o.cache_append(b.cfg, d[:, :8], d[:, 8:10], d[:, 10:], kc, vc, b.table.cuda(), b.q_start.cuda(),
                           b.kv_len.cuda(), rotary=r, positions=None if pos is None else pos.cuda(), q_out=q_out)
    assert got is q_out and s2o.last_launch_count() == 1 and s2o.last_device_error() == 0
    at = np.concatenate([np.arange(L - n, L) for n, L in zip(new, length)])
    p = np.tile(at + P, (axes, 1)) if pos is None else pos.numpy()[:, :b.own]
    x = f64(qkv)[:b.own]
    wq, mq = SO.rotate(x[:, :8], p, 128, r.axis, r.inv_freq, adjacent)
    wk, mk = SO.rotate(x[:, 8:10], p, 128, r.axis, r.inv_freq, adjacent)
    assert_rotated(q_out[:b.own], wq, mq, t)
    assert bool((q_out[b.own:] == 3.0).all())
    seq = np.concatenate([np.full(n, s) for s, n in enumerate(new)]).astype(int)
    pg = b.table.numpy()[seq, at // page]
    assert_rotated(kc[pg, :, at % page], wk, mk, t)
    assert torch.equal(vc[pg, :, at % page].cpu(), qkv[:b.own, 10:])
    # nothing else moved (bit patterns: the rest holds NaN)
    for c, c0 in ((kc, k0), (vc, v0)):
        c = c.cpu().view(torch.int16)
        c[pg, :, at % page] = c0.view(torch.int16)[pg, :, at % page]
        assert torch.equal(c, c0.view(torch.int16))


def test_append_without_rotation_and_without_queries():
    b = Batch([3, 2], [20, 2])
    x = torch.randn(5, 2, 128, device="cuda").bfloat16()
    kc, vc = b.k.cuda(), b.v.cuda()
    assert s2o.cache_append(b.cfg, None, x, 2 * x, kc, vc, b.table.cuda(), b.q_start.cuda(), b.kv_len.cuda()) is None
    assert s2o.last_device_error() == 0
    pages = b.table[[0, 0, 0, 1, 1], [1, 1, 1, 0, 0]].long()
    rows = torch.tensor([1, 2, 3, 0, 1])
    assert torch.equal(kc[pages, :, rows], x) and torch.equal(vc[pages, :, rows], 2 * x)


def test_append_flags_bad_pages_and_lengths_and_writes_nothing_there():
    for what in ("page high", "page negative", "length", "short", "start", "many"):
        b = Batch([2, 2], [18, 9])
        table, qs, kl = b.table.clone(), b.q_start.clone(), b.kv_len.clone()
        if what == "page high":
            table[0, 1] = b.cfg.num_pages
        elif what == "page negative":
            table[0, 1] = -1
        elif what == "length":
            kl[0] = b.cfg.max_pages * 16 + 1
        elif what == "short":
            kl[0] = 1
        elif what == "start":
            qs[1] = 5
        else:
            qs[1:] = 3
        x = torch.randn(4, 2, 128, device="cuda").bfloat16()
        kc, vc = b.k.cuda(), b.v.cuda()
        s2o.cache_append(b.cfg, None, x, x, kc, vc, table.cuda(), qs.cuda(), kl.cuda())
        assert s2o.last_device_error() == BAD_CACHE, what
        assert s2o.last_device_error() == 0
        own0 = b.table[0, :2].long()
        assert torch.equal(kc.cpu()[own0].view(torch.int16), b.k[own0].view(torch.int16)), what


def test_append_flags_ranges_that_none_of_its_tokens_leads_to():
    """A sequence that lies behind the rows, descending starts, starts that do not
    begin at 0, one bad entry among hundreds of sequences without tokens: flagged
    as the attention flags them, and cache rows of nobody stay."""
    for qs, kl in (([0, 4, 1000], [9, 9]), ([0, 4, 2], [9, 9]), ([0, 0, -1], [9, 9]), ([2, 2, 2], [9, 9]),
                   ([0, 2, 4] + [4] * 298 + [6], [9] * 301), ([0] * 200 + [-3] + [0] * 100 + [4], [9] * 301)):
        nseq = len(kl)
        b = Batch([4] + [0] * (nseq - 1), [9] * nseq, max_q=8)
        qs, kl, table = (torch.tensor(x, dtype=torch.int32).cuda() for x in (qs, kl, b.table.tolist()))
        x = torch.randn(4, 2, 128, device="cuda").bfloat16()
        kc, vc = b.k.cuda(), b.v.cuda()
        s2o.cache_append(b.cfg, None, x, x, kc, vc, table, qs, kl)
        assert s2o.last_device_error() == BAD_CACHE, qs.tolist()[:4]
        free = [i for i in range(b.cfg.num_pages) if i not in b.table.flatten().tolist()]
        assert torch.equal(kc.cpu()[free].view(torch.int16), b.k[free].view(torch.int16))
        s2o.attention_paged(b.cfg, torch.zeros(4, 8, 128, device="cuda").bfloat16(), torch.nan_to_num(kc),
                            torch.nan_to_num(vc), table, qs, kl)
        assert s2o.last_device_error() == BAD_CACHE, qs.tolist()[:4]
    b = Batch([0] * 150 + [4] + [0] * 150, [9] * 301)  # sequences without tokens need no length
    kl = torch.where(torch.arange(301) == 150, 9, -7).int().cuda()
    kc, vc = b.k.cuda(), b.v.cuda()
    s2o.cache_append(b.cfg, None, x, x, kc, vc, b.table.cuda(), b.q_start.cuda(), kl)
    assert s2o.last_device_error() == 0
    assert torch.equal(kc[b.table[150, 0].long(), :, 5:9], x.transpose(0, 1))


# --- attention ----------------------------------------------------------------------------------------

CASES = {
    # new tokens, own keys, prefix, page, Hq, Hkv
    "one_key": ([1], [1], 0, 16, 8, 2),
    "tile_edges": ([1] * 8, [1, 15, 16, 17, 63, 64, 65, 129], 0, 16, 8, 2),
    "prefix_one_key": ([1, 1], [1, 2], 1, 16, 8, 2),
    "prefix_ends_in_page": ([1] * 4, [1, 40, 64, 200], 77, 32, 8, 2),
    "prefix_edges": ([1] * 3, [3, 3, 3], 128, 64, 8, 8),
    "no_sharing": ([1] * 3, [300, 1, 64], 200, 128, 3, 3),
    "empty_sequences": ([0, 1, 0, 3, 0], [9, 50, 0, 70, 64], 90, 16, 8, 2),
    "drafts": ([5] * 6, [5, 6, 64, 65, 130, 400], 100, 32, 16, 2),
    "drafts_ragged": ([1, 7, 2, 9], [100, 7, 3, 61], 0, 64, 12, 4),
    "group_of_3": ([1, 2, 17], [30, 2, 90], 50, 16, 3, 1),
    "group_of_40": ([1, 3], [70, 140], 65, 16, 40, 1),
    "group_of_64": ([1, 2], [70, 5], 130, 16, 64, 1),
    "many_rows": ([1] * 70, [1 + 3 * i for i in range(70)], 333, 16, 8, 2),
    "chunk": ([130, 1, 70], [130, 60, 200], 150, 64, 8, 2),
    "chunk_alone": ([200], [200], 0, 128, 4, 1),
    "chunks_no_group": ([40, 33], [140, 33], 20, 16, 2, 2),
    "long_one": ([1], [3000], 0, 16, 2, 2),
    "long_prefix": ([1, 1], [5, 9], 4099, 128, 4, 1),
    "wide_chunk": ([300, 257], [301, 900], 129, 32, 16, 4),
}


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(CASES))
def test_attention_matches_the_oracle(name, t):
    new, length, P, page, Hq, Hkv = CASES[name]
    b = Batch(new, length, P, page, Hq, Hkv, TYPES[t], seed=len(name), extra_rows=2)
    # outputs and workspace poisoned: what is not written shows, rows of nobody stay
    O = torch.full((b.Tq, Hq, 128), 5.0, device="cuda", dtype=TYPES[t])
    lse = torch.full((b.Tq, Hq), 5.0, device="cuda")
    ws = s2o.alloc_attention_paged(b.cfg).fill_(255)
    got, gl = attend(b, O=O, lse=lse, workspace=ws)
    assert got is O and gl is lse
    b.check(O, lse, name)
    assert bool((O[b.own:] == 5.0).all()) and bool((lse[b.own:] == 5.0).all())
    O2, lse2 = attend(b, workspace=ws)
    assert torch.equal(O2[:b.own], O[:b.own]) and torch.equal(lse2[:b.own], lse[:b.own])  # no atomics: the same bits
    O32, _ = attend(b, out_dtype=s2o.OUT_F32)
    assert O32.dtype == torch.float32
    b.check(O32, None, name + " fp32")


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_attention_with_large_scores(t):
    """Scores of some hundreds: the reference moves many times, all the mass sits
    on few keys."""
    for seed in range(3):
        attend_b = Batch([1, 3, 80], [500, 90, 100], 600, 16, 8, 2, TYPES[t], seed=seed, scale=5.0)
        O, lse = attend(attend_b)
        attend_b.check(O, lse, seed)


def test_a_rising_and_a_falling_run_of_scores():
    """Keys in order of rising scores rescale at every tile, falling ones never."""
    for sign in (1.0, -1.0):
        b = Batch([1, 4], [700, 700], 300, 64, 8, 2, torch.float16)
        ramp = torch.linspace(-12, 12, 1000) * sign
        u = torch.ones(128) / 128 ** 0.5
        for pages, n, first in ((b.prefix_pages, 300, 0), (b.table[0], 700, 300), (b.table[1], 700, 300)):
            for i in range(n):
                b.k[pages[i // 64], :, i % 64] = (b.k[pages[i // 64], :, i % 64].float() * 0.1 + ramp[first + i] * u).half()
        b.q = (b.q.float() * 0.1 + 11.0 * u).half()
        O, lse = attend(b)
        b.check(O, lse, sign)


def dense_reference(b, q, k, v, table, kv_len, prefix_pages):
    """SO.attend for batches too large for it: the same in fp64 with torch on the
    GPU, a sequence at a time."""
    Tq, Hq, Hkv, d = q.shape[0], q.shape[1], k.shape[1], 128
    G, P = Hq // Hkv, b.P
    rows = lambda c, pages, n: c[pages.long()].transpose(1, 2).reshape(-1, Hkv, d)[:n].double()
    O, A = (torch.zeros(Tq, Hq, d, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, S = (torch.zeros(Tq, Hq, dtype=torch.float64, device="cuda") for _ in range(2))
    n = torch.zeros(Tq, dtype=torch.int64)
    pk, pv = rows(k, prefix_pages, P), rows(v, prefix_pages, P)
    t0 = 0
    for s, (m, L) in enumerate(zip(b.new, b.len)):
        if m:
            used = table[s, :-(-L // b.page)]
            kk = torch.cat([pk, rows(k, used, L)]).permute(1, 2, 0)                  # [Hkv, d, n]
            vv = torch.cat([pv, rows(v, used, L)]).transpose(0, 1)                   # [Hkv, n, d]
            qq = q[t0:t0 + m].double().view(m, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, G * m, d)
            x = (qq @ kk).view(Hkv, G, m, -1) / d ** 0.5
            key = torch.arange(P + L, device="cuda")
            at = P + L - m + torch.arange(m, device="cuda")
            hidden = key[None] > at[:, None]
            x = x.masked_fill(hidden, float("-inf")).view(Hkv, G * m, -1)
            p = torch.softmax(x, -1)
            back = lambda y: y.view(Hkv, G, m, -1).permute(2, 0, 1, 3).reshape(m, Hq, -1)
            O[t0:t0 + m], A[t0:t0 + m] = back(p @ vv), back(p @ vv.abs())
            lse[t0:t0 + m] = back(torch.logsumexp(x, -1)[..., None])[..., 0]
            S[t0:t0 + m] = back((qq.abs() @ kk.abs()).amax(-1, keepdim=True))[..., 0] / d ** 0.5
            n[t0:t0 + m] = (at + 1).cpu()
        t0 += m
    return f64(O), f64(lse), f64(A), f64(S), n.numpy()


# shapes that reach every way the kernels are put together: (new, own keys, prefix, page, Hq, Hkv, launches)
WAYS = {
    "decode_walks_prefix": ([1] * 40, [1 + 7 * i % 300 for i in range(40)], 40, 16, 32, 8, 2),
    "decode_two_row_tiles": ([3, 8, 5] * 5, [20, 8, 400] * 5, 0, 32, 16, 4, 2),
    "decode_prefix_items": ([1] * 24, [1 + 11 * i % 200 for i in range(24)], 5000, 64, 8, 2, 2),
    "tiles_in_teams": ([1] * 200, [1 + i % 90 for i in range(200)], 4100, 64, 32, 8, 3),
    "tiles_in_teams_ragged": ([2, 0, 4, 1] * 60, [70, 3, 4, 31] * 60, 9001, 128, 8, 2, 3),
    "tiles_without_teams": ([1] * 700, [1 + i % 40 for i in range(700)], 3000, 16, 32, 1, 3),
    "tiles_of_128_rows": ([1] * 30, [1 + i % 60 for i in range(30)], 30000, 32, 8, 2, 3),
    "chunks_walk_prefix": ([100, 33, 260], [100, 400, 900], 700, 32, 8, 2, 2),
    "chunks_prefix_items": ([9] * 64, [9 + 5 * i for i in range(64)], 6000, 16, 32, 8, 2),
    "chunks_alone_long": ([1500], [2600], 0, 128, 4, 1, 2),
    "chunk_groups_of_48": ([1, 2, 9], [100, 2, 300], 500, 64, 48, 1, 2),
}


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("way", list(WAYS))
def test_every_way_of_the_attention(way, t):
    new, length, P, page, Hq, Hkv, launches = WAYS[way]
    b = Batch(new, length, P, page, Hq, Hkv, TYPES[t], seed=11, extra_rows=1)
    q, k, v, table, qs, kl, pre = b.dev()
    ws = s2o.alloc_attention_paged(b.cfg).fill_(255)
    O, lse = s2o.attention_paged(b.cfg, q, k, v, table, qs, kl, prefix_pages=pre, workspace=ws)
    assert s2o.last_launch_count() == launches
    assert s2o.last_device_error() == 0
    b.want = dense_reference(b, q, k, v, table, kl, pre)
    b.check(O, lse, way)
    # called again and again, other work of the same kernels in between: the same bits
    c = Batch([1, 40], [77, 90], 300, 16, 8, 2, TYPES[t], seed=12)
    for _ in range(10):
        O2, lse2 = s2o.attention_paged(b.cfg, q, k, v, table, qs, kl, prefix_pages=pre, workspace=ws)
        attend(c)
        assert torch.equal(O2[:b.own], O[:b.own]) and torch.equal(lse2[:b.own], lse[:b.own])


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_equal_chunks_walk_the_prefix(t):
    """Chunks of equal length go tile by tile through prefix and own keys: two
    launches, no second list of parts."""
    b = Batch([64] * 16, [64 + 31 * i for i in range(16)], 8190, 64, 8, 2, TYPES[t], seed=21, extra_rows=1)
    assert ways.way(b.cfg) == "chunks walk"
    q, k, v, table, qs, kl, pre = b.dev()
    ws = s2o.alloc_attention_paged(b.cfg).fill_(255)
    O, lse = s2o.attention_paged(b.cfg, q, k, v, table, qs, kl, prefix_pages=pre, workspace=ws)
    assert s2o.last_launch_count() == 2 and s2o.last_device_error() == 0
    b.want = dense_reference(b, q, k, v, table, kl, pre)
    b.check(O, lse)


# the decode kernel with two row tiles and the prefix in its own streams: both key lists in one piece, their
# border anywhere in a stage ring; (new, own keys, prefix, page, Hq, Hkv, way)
TWO_ROW_TILES = {
    "walk_drafts_of_8": ([5, 8, 6], [40, 8, 177], 77, 16, 32, 8, "decode2 walk"),
    "walk_ragged": ([8, 1, 3, 0] * 8, [61, 500, 3, 90] * 8, 201, 64, 8, 2, "decode2 walk"),
    "walk_one_key": ([5] * 6, [5, 6, 64, 65, 130, 400], 1, 16, 8, 2, "decode2 walk"),
    "walk_group_of_20": ([1] * 9, [1 + 40 * i for i in range(9)], 499, 32, 40, 2, "decode2 walk"),
    "walk_group_of_12": ([1, 2] * 6, [33, 64] * 6, 90, 128, 24, 2, "decode2 walk"),
    "items": ([8] + [1] * 20, [9] + [1 + 17 * i for i in range(20)], 1001, 32, 8, 2, "decode2 items"),
    "items_32_heads": ([7] + [1] * 20, [300] + [1 + 9 * i for i in range(20)], 1009, 64, 32, 8, "decode2 items"),
}


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("name", list(TWO_ROW_TILES))
def test_two_row_tiles_with_the_prefix_in_the_same_kernel(name, t):
    new, length, P, page, Hq, Hkv, way = TWO_ROW_TILES[name]
    b = Batch(new, length, P, page, Hq, Hkv, TYPES[t], seed=31, extra_rows=2)
    assert ways.way(b.cfg) == way
    O = torch.full((b.Tq, Hq, 128), 5.0, device="cuda", dtype=TYPES[t])
    lse = torch.full((b.Tq, Hq), 5.0, device="cuda")
    ws = s2o.alloc_attention_paged(b.cfg).fill_(255)
    attend(b, O=O, lse=lse, workspace=ws)
    assert s2o.last_launch_count() == 2
    b.check(O, lse, name)
    assert bool((O[b.own:] == 5.0).all()) and bool((lse[b.own:] == 5.0).all())
    for _ in range(5):
        O2, lse2 = attend(b, workspace=ws)
        assert torch.equal(O2[:b.own], O[:b.own]) and torch.equal(lse2[:b.own], lse[:b.own])


def test_a_batch_without_tokens():
    """No token at all, or rows that belong to nobody: nothing is written."""
    b = Batch([0, 0], [30, 0], 40)
    x = torch.zeros(0, 8, 128, device="cuda").bfloat16()
    q, k, v, table, qs, kl, pre = b.dev()
    O, lse = s2o.attention_paged(b.cfg, q, k, v, table, qs, kl, prefix_pages=pre)
    assert O.shape == (0, 8, 128) and s2o.last_launch_count() == 0
    s2o.cache_append(b.cfg, x, x[:, :2], x[:, :2], k, v, table, qs, kl, rotary=s2o.make_rotary())
    assert s2o.last_launch_count() == 0
    assert s2o.rotary(s2o.make_rotary(), x[None], None, torch.zeros(1, 1, 0, device="cuda", dtype=torch.int32))[0].numel() == 0
    for P in (0, 40, 5000):
        b = Batch([0, 0], [30, 0], P, extra_rows=70)
        O = torch.full((70, 8, 128), 5.0, device="cuda", dtype=torch.bfloat16)
        attend(b, O=O)
        assert bool((O == 5.0).all())
        q, k, v, table, qs, kl, pre = b.dev()
        before = k.view(torch.int16).clone()
        y = torch.ones(70, 2, 128, device="cuda").bfloat16()
        s2o.cache_append(b.cfg, None, y, y, k, v, table, qs, kl)
        assert torch.equal(k.view(torch.int16), before) and s2o.last_device_error() == 0


def test_lse_may_be_left_out_and_the_workspace_must_fit():
    b = Batch([1, 1], [30, 9], 40)
    q, k, v, table, qs, kl, pre = b.dev()
    ws = s2o.alloc_attention_paged(b.cfg)
    O = torch.empty_like(q)
    p = lambda x: x.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    args = [b.cfg, p(q), p(k), p(v), p(pre), p(table), p(qs), p(kl), p(O), 0, None, p(ws), ws.numel(), stream]
    assert s2o.lib().s2o_attention_paged(*args) == 0
    assert s2o.last_device_error() == 0
    b.check(O, None)
    with pytest.raises(s2o.S2OError) as e:
        s2o.attention_paged(b.cfg, q, k, v, table, qs, kl, prefix_pages=pre, workspace=ws[:ws.numel() - 256])
    assert e.value.code == 3


def test_attention_flags_bad_pages_lengths_and_ranges():
    for what in ("page high", "page negative", "prefix page", "length", "short", "descending", "start", "many", "rows"):
        b = Batch([2, 2], [40, 9], 20)
        q, k, v, table, qs, kl, pre = b.dev()
        k, v = torch.nan_to_num(k), torch.nan_to_num(v)
        if what == "page high":
            table[0, 1] = b.cfg.num_pages
        elif what == "page negative":
            table[0, 0] = -7
        elif what == "prefix page":
            pre[1] = 1 << 30
        elif what == "length":
            kl[0] = 1 << 30
        elif what == "short":
            kl[0] = 1
        elif what == "descending":
            qs[1] = 4
            qs[2] = 2
        elif what == "start":
            qs[0] = 1
        elif what == "many":
            qs[1] = 3
        else:
            qs[2] = 1000
        s2o.attention_paged(b.cfg, q, k, v, table, qs, kl, prefix_pages=pre)
        assert s2o.last_device_error() == BAD_CACHE, what
        assert s2o.last_device_error() == 0, what
    b = Batch([2, 2], [40, 9], 20)  # and a good call afterwards is right
    b.check(*attend(b))


def test_another_stream_and_captured_calls_follow_the_arrays():
    b = Batch([1, 1, 1], [100, 33, 64], 150, 16, 8, 2)
    q, k, v, table, qs, kl, pre = b.dev()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    O, lse = s2o.attention_paged(b.cfg, q, k, v, table, qs, kl, prefix_pages=pre, stream=side)
    assert s2o.last_device_error(side) == 0
    b.check(O, lse, "side stream")
    # two graphs of the same shapes, a workspace each, replayed in turn and side by side
    ws = [s2o.alloc_attention_paged(b.cfg) for _ in range(2)]
    outs = [(torch.zeros_like(q), torch.zeros(3, 8, device="cuda")) for _ in range(2)]
    lens = [kl.clone(), kl.clone()]
    graphs = []
    for w, (o, l), n in zip(ws, outs, lens):
        s2o.attention_paged(b.cfg, q, k, v, table, qs, n, prefix_pages=pre, O=o, lse=l, workspace=w)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            s2o.attention_paged(b.cfg, q, k, v, table, qs, n, prefix_pages=pre, O=o, lse=l, workspace=w)
        graphs.append(gr)
    for lengths in ([100, 33, 64], [7, 1, 50], [64, 32, 1]):
        lens[1].copy_(torch.tensor(lengths, dtype=torch.int32))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert s2o.last_device_error() == 0
        b.check(*outs[0], "graph 0")
        c = Batch([1, 1, 1], [100, 33, 64], 150, 16, 8, 2)
        c.kv_len = torch.tensor(lengths, dtype=torch.int32)
        c.check(*outs[1], lengths)


def test_rows_beyond_32_bits_of_elements():
    """A cache of over 2^31 elements, the sequence's pages at its end."""
    page, Hkv = 128, 8
    num_pages = (1 << 31) // (page * Hkv * 128) + 9
    b = Batch([1, 2], [300, 200], 130, page, 16, Hkv, seed=4)
    k, v = (torch.zeros(num_pages, Hkv, page, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    shift = num_pages - b.cfg.num_pages
    k[shift:], v[shift:] = b.k.cuda(), b.v.cuda()
    b.cfg.num_pages = num_pages
    table = torch.where(b.table >= 0, b.table + shift, -1).int().cuda()
    qs, kl, q = b.q_start.cuda(), b.kv_len.cuda(), b.q.cuda()
    x = torch.randn(3, 2 * Hkv, 128, device="cuda").bfloat16()
    s2o.cache_append(b.cfg, None, x[:, :Hkv], x[:, Hkv:], k, v, table, qs, kl)
    b.k, b.v = k[shift:].cpu(), v[shift:].cpu()
    O, lse = s2o.attention_paged(b.cfg, q, k, v, table, qs, kl, prefix_pages=(b.prefix_pages + shift).int().cuda())
    assert s2o.last_device_error() == 0
    pg = b.table[[0, 1, 1], [2, 1, 1]].long()
    assert torch.equal(b.k[pg, :, torch.tensor([43, 70, 71])], x[:, :Hkv].cpu())
    b.check(O, lse)


def test_prompt_then_steps_as_a_program_runs_them():
    """rotary -> plan + attention (the prefill, tau = 0: exact) -> append ->
    steps of append + attention_paged, each against dense attention in fp64."""
    N, Hq, Hkv, page, steps, S = 300, 4, 2, 32, 3, 2
    P, own = 256, N - 256  # the prompt's first 256 tokens are the shared prefix
    Q, K, V = synth.generate(1, Hq, Hkv, N, 128, planted=True, band=False, n_stripe=4, seed=5)
    bf = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)[0].transpose(0, 1).cuda()
    q, k, v = bf(Q), bf(K), bf(V)  # [N, H, 128], head-major memory
    r = s2o.make_rotary(128, theta=500000.0)
    pos = torch.arange(N, device="cuda", dtype=torch.int32)
    qr, kr = s2o.rotary(r, q[None], k[None], pos.view(1, 1, N))
    qh, kh, vh = qr.transpose(1, 2), kr.transpose(1, 2), v.transpose(0, 1)[None].contiguous()
    cfg = s2o.make_config(1, Hq, Hkv, N, tau=0.0)
    bufs = s2o.plan(cfg, qh, kh)
    out = s2o.attention(cfg, qh, kh, vh, bufs["perm"], bufs["nblocks"])  # [1, Hq, N, 128]
    assert s2o.last_device_error() == 0

    num_pages = P // page + S * 4
    make = lambda **kw: s2o.make_cache(Hq, Hkv, page, num_pages, max_pages=4, **kw)
    kc, vc = s2o.alloc_cache(make(nseq=1, Tq=1))
    pre = torch.arange(P // page, device="cuda", dtype=torch.int32)
    table = (P // page + torch.arange(S * 4, device="cuda", dtype=torch.int32)).view(S, 4)
    i32 = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)
    # the prefix: one sequence of its own pages (rotated already)
    wide = s2o.make_cache(Hq, Hkv, page, num_pages, nseq=1, max_pages=P // page, Tq=P, max_q=P)
    s2o.cache_append(wide, None, kr[0, :P], v[:P], kc, vc, pre.view(1, -1), i32(0, P), i32(P))
    # the rest of the prompt, in both sequences, rotated by the append itself
    rest = make(nseq=S, Tq=S * own, max_q=own, prefix_len=P)
    two = lambda x: torch.cat([x[P:], x[P:]])
    starts = i32(0, own, 2 * own)
    q2 = s2o.cache_append(rest, two(q), two(k), two(v), kc, vc, table, starts, i32(own, own), rotary=r)
    assert torch.equal(q2[:own], qr[0, P:]) and torch.equal(q2[own:], qr[0, P:])
    chunk, _ = s2o.attention_paged(rest, q2, kc, vc, table, starts, i32(own, own), prefix_pages=pre)
    assert s2o.last_device_error() == 0

    def dense(qrow, keys, vals):  # [Hq, d], [n, Hkv, d]
        o = np.zeros((Hq, 128))
        a = np.zeros((Hq, 128))
        for h in range(Hq):
            x = keys[:, h // 2] @ qrow[h] / np.sqrt(128)
            p = np.exp(x - x.max())
            o[h], a[h] = p @ vals[:, h // 2] / p.sum(), p @ np.abs(vals[:, h // 2]) / p.sum()
        return o, a

    u = half_step(torch.bfloat16)
    kd, vd, qd = f64(kr[0]), f64(v), f64(qr[0])
    for t in (P, P + 1, N - 1):
        o, a = dense(qd[t], kd[:t + 1], vd[:t + 1])
        tol = u * np.abs(o) + 1.1 * u * a  # score and sum errors: below a tenth of P's rounding at 300 keys
        assert (np.abs(f64(out[0, :, t]) - o) <= tol).all()
        for s in range(S):
            assert (np.abs(f64(chunk[s * own + t - P]) - o) <= tol).all()

    step = make(nseq=S, Tq=S, prefix_len=P)
    ws = s2o.alloc_attention_paged(step)
    g = torch.Generator(device="cuda").manual_seed(1)
    seen = [(kd, vd)] * S
    for n in range(steps):
        qkv = torch.randn(S, Hq + 2 * Hkv, 128, generator=g, device="cuda").bfloat16()
        kl = i32(own + n + 1, own + n + 1)
        qn = s2o.cache_append(step, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kc, vc, table, i32(0, 1, 2), kl,
                              rotary=r)
        O, _ = s2o.attention_paged(step, qn, kc, vc, table, i32(0, 1, 2), kl, prefix_pages=pre, workspace=ws)
        assert s2o.last_device_error() == 0
        kn, _ = SO.rotate(f64(qkv[:, Hq:Hq + Hkv]), np.full((1, S), N + n), 128, r.axis, r.inv_freq)
        kn = torch.from_numpy(kn).bfloat16().double().numpy()
        for s in range(S):
            at = own + n
            row = f64(kc[table[s, at // page], :, at % page])  # the cached key: the rotated one, to a rounding
            assert (np.abs(row - kn[s]) <= 2 * u * np.abs(kn[s]) + 1e-5).all()
            seen[s] = (np.concatenate([seen[s][0], row[None]]),
                       np.concatenate([seen[s][1], f64(qkv[s:s + 1, Hq + Hkv:])]))
            o, a = dense(f64(qn[s]), *seen[s])
            assert (np.abs(f64(O[s]) - o) <= u * np.abs(o) + 1.1 * u * a).all()
