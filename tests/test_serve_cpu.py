"""The serving calls without a GPU: the oracle's own pins, every refusal that
is made before a launch, and the host-side arithmetic of the configs."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

import score_keys_pooled_b200 as s2o
from score_keys_pooled_b200 import build
from oracle import serve_oracle as SO
from tests import serve_ways as ways

GOOD = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def L():
    build.build()
    return s2o.lib()


def cache(**kw):
    c = dict(Hq=8, Hkv=2, page_size=16, num_pages=10, nseq=2, max_pages=4, Tq=3, max_q=2, prefix_len=20)
    c.update(kw)
    return s2o.make_cache(**c)


def view(ptr=1 << 20, b=0, t=1024, h=128):
    return ctypes.byref(s2o.View(ptr, b, t, h))


def test_oracle_rotation_is_complex_multiplication_and_inverts():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 3, 128)), np.array([[0, 1, 7, 1000, 12345]])
    freq = 10000.0 ** (-np.arange(32) / 32.0)
    y, _ = SO.rotate(x, pos, 64, [0] * 32, freq)
    z = (x[:, :, :32] + 1j * x[:, :, 32:64]) * np.exp(1j * pos[0][:, None, None] * freq)
    assert np.allclose(y[:, :, :32], z.real, atol=1e-12) and np.allclose(y[:, :, 32:64], z.imag, atol=1e-12)
    assert np.array_equal(y[:, :, 64:], x[:, :, 64:]) and np.array_equal(y[0], x[0])
    assert np.allclose(SO.rotate(y, pos, 64, [0] * 32, freq, inverse=True)[0], x, atol=1e-12)


def test_oracle_inverse_is_the_gradient():
    """<g, d rotate(x)/dx_i> by central differences (the map is linear: exact)."""
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((2, 1, 128)), rng.standard_normal((2, 1, 128))
    pos = np.array([[3, 900], [5, 1], [0, 77]])
    r = s2o.make_rotary(96, sections=(12, 18, 18), interleaved=True)
    turn = lambda y, inv=False: SO.rotate(y, pos, 96, r.axis, r.inv_freq, True, inv)[0]
    back = turn(g, True)
    for i in (0, 1, 30, 95, 96, 127):
        e = np.zeros_like(x)
        e[:, :, i] = 0.5
        diff = ((turn(x + e) - turn(x - e)) * g).sum((1, 2))
        assert np.allclose(diff, back[:, 0, i], atol=1e-12)


def test_oracle_attention_is_one_softmax_over_prefix_and_own_keys():
    rng = np.random.default_rng(2)
    kc, vc = rng.standard_normal((6, 2, 16, 128)), rng.standard_normal((6, 2, 16, 128))
    q = rng.standard_normal((3, 4, 128))
    O, lse, _, _, n = SO.attend(q, kc, vc, np.array([[4, 1]]), [0, 3], [19], [5, 0], 17)
    k = np.concatenate([kc[5, 1], kc[0, 1, :1], kc[4, 1], kc[1, 1, :2]])  # token 1 sees 17 + 18 of 19 own keys
    v = np.concatenate([vc[5, 1], vc[0, 1, :1], vc[4, 1], vc[1, 1, :2]])
    p = np.exp(k @ q[1, 2] / np.sqrt(128))
    assert list(n) == [34, 35, 36] and np.allclose(lse[1, 2], np.log(p.sum()))
    assert np.allclose(O[1, 2], p @ v / p.sum())


def test_a_packed_view_is_a_view():
    v = s2o.View(1 << 40, 3, -8, 1 << 33)
    assert bytes(v) == s2o._pack_view(1 << 40, 3, -8, 1 << 33)


def test_rotary_config_checks():
    r = s2o.make_rotary(64, theta=500.0, sections=(8, 10, 14))
    assert list(r.axis[:32]) == [0] * 8 + [1] * 10 + [2] * 14 and r.naxes == 3
    assert r.inv_freq[5] == 500.0 ** (-10 / 64)
    for kw in (dict(rot_dim=130), dict(rot_dim=-2), dict(rot_dim=63), dict(sections=(1, 2)),
               dict(sections=(16, 16, 16, 16)), dict(sections=(65, -1)), dict(inv_freq=[1.0])):
        with pytest.raises(s2o.S2OError):
            s2o.make_rotary(**kw)


@pytest.mark.parametrize("change,code", [
    (dict(Hq=0), 1), (dict(Hkv=3), 1), (dict(nseq=0), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1),
    (dict(Tq=-1), 1), (dict(max_q=0), 1), (dict(prefix_len=-1), 1), (dict(dtype=2), 1), (dict(d=64), 2),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=256), 2), (dict(Hq=130, Hkv=2), 2),
    (dict(num_pages=1 << 27, page_size=16), 2), (dict(max_pages=1 << 27), 2), (dict(Tq=1 << 28), 2),
])
def test_cache_config_validation(L, change, code):
    c = cache(**change)
    n = ctypes.c_size_t(0)
    assert L.s2o_attention_paged_workspace_size(c, n) == code
    assert L.s2o_attention_paged(c, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, 0, None, GOOD, 1 << 40, None) == code
    assert L.s2o_cache_append(c, None, None, view(), view(), None, GOOD, GOOD, GOOD, GOOD, GOOD, None, None) == code
    assert s2o.last_launch_count() == 0


@pytest.mark.parametrize("nseq,max_q,Tq,prefix,heads,want,mb", [
    # equal chunks: the row tiles of the walk are those of the items, which join a second list
    (32, 64, 32 * 64, 32768, (32, 8), "chunks walk", 39.1), (16, 256, 16 * 256, 32768, (32, 8), "chunks walk", 39.1),
    (8, 128, 8 * 128, 16384, (32, 8), "chunks walk", 39.1), (16, 64, 16 * 64, 8192, (32, 8), "chunks walk", 39.1),
    # one chunk among single tokens: the host knows 64 + floor(511 / 64) tiles at most
    (64, 512, 512 + 63, 8192, (32, 8), "chunks items", 58.4),
    (20, 40, 800, 1500, (8, 8), "chunks items", 46.1), (33, 5, 165, 5001, (16, 2), "chunks items", 42.0),
    (16, 4, 64, 1000, (32, 8), "decode1 tiles", 61.0), (32, 5, 160, 8192, (32, 8), "decode2 tiles", 64.0),
    (16, 1, 16, 20000, (32, 8), "decode1 tiles", None), (1, 1, 1, 1024, (32, 8), "decode1 walk", None),
    (1, 1, 1, 0, (32, 8), "decode1 walk", None),
])
def test_the_way_of_the_prefix(L, nseq, max_q, Tq, prefix, heads, want, mb):
    c = s2o.make_cache(*heads, page_size=64, num_pages=4096, nseq=nseq, max_pages=40, Tq=Tq, max_q=max_q,
                       prefix_len=prefix)
    assert ways.way(c) == want
    if mb:
        assert abs(ways.sizes(c)[want] / 1e6 - mb) < 1.0


def test_the_gpu_tests_reach_the_ways_they_name(L):
    from tests.test_serve import WAYS
    want = {"decode_walks_prefix": "decode1 walk", "decode_two_row_tiles": "decode2 walk",
            "decode_prefix_items": "decode1 items", "tiles_in_teams": "decode1 tiles",
            "tiles_in_teams_ragged": "decode1 tiles", "tiles_without_teams": "decode2 tiles",
            "tiles_of_128_rows": "decode1 tiles", "chunks_walk_prefix": "chunks walk",
            "chunks_prefix_items": "chunks items", "chunks_alone_long": "chunks walk",
            "chunk_groups_of_48": "chunks walk"}
    for name, (new, length, P, page, Hq, Hkv, _) in WAYS.items():
        c = s2o.make_cache(Hq, Hkv, page, 1 << 14, len(new), max(1, max(length) // page + 1), sum(new) + 1,
                           max_q=max(new), prefix_len=P)
        assert ways.way(c) == want[name], name


def test_attention_paged_refusals(L):
    c = cache()
    need = s2o.attention_paged_workspace_size(c)
    good = [c, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, ctypes.c_void_p(1 << 21), 0, None, GOOD, need, None]
    for i in (1, 2, 3, 4, 5, 6, 7, 8, 11):
        assert L.s2o_attention_paged(*(good[:i] + [None] + good[i + 1:])) == 1, i
    for i in (1, 2, 3, 8, 11):
        assert L.s2o_attention_paged(*(good[:i] + [ODD] + good[i + 1:])) == 1, i
    assert L.s2o_attention_paged(*(good[:9] + [2] + good[10:])) == 1
    assert L.s2o_attention_paged(*(good[:8] + [ctypes.c_void_p(1 << 20)] + good[9:])) == 1  # O in Q's place
    assert L.s2o_attention_paged(*(good[:12] + [need - 1, None])) == 3
    assert L.s2o_attention_paged_workspace_size(c, None) == 1
    empty = cache(Tq=0)
    assert L.s2o_attention_paged(*([empty] + good[1:])) == 0 and s2o.last_launch_count() == 0


def test_append_refusals(L):
    c, r = cache(), s2o.make_rotary(128)
    good = [c, r, view(), view(), view(), None, GOOD, GOOD, GOOD, GOOD, GOOD, view(), None]
    for i in (2, 3, 4, 6, 7, 8, 9, 10, 11):  # q and q_out come together
        assert L.s2o_cache_append(*(good[:i] + [None] + good[i + 1:])) == 1, i
    for i in (9, 10):
        assert L.s2o_cache_append(*(good[:i] + [ODD] + good[i + 1:])) == 1, i
    for i in (2, 3, 4, 11):
        for bad in (view(ptr=(1 << 20) + 2), view(t=1028), view(h=4), view(ptr=0)):
            assert L.s2o_cache_append(*(good[:i] + [bad] + good[i + 1:])) == 1, i
    bad = s2o.make_rotary(128)
    for field, value, code in (("rot_dim", 24, 2), ("rot_dim", 144, 2), ("rot_dim", -16, 1), ("naxes", 0, 1),
                               ("naxes", 4, 1)):
        b = s2o.make_rotary(128)
        setattr(b, field, value)
        assert L.s2o_cache_append(*(good[:1] + [b] + good[2:])) == code
    bad.inv_freq[3] = float("nan")
    assert L.s2o_cache_append(*(good[:1] + [bad] + good[2:])) == 1
    bad = s2o.make_rotary(128)
    bad.axis[7] = 1
    assert L.s2o_cache_append(*(good[:1] + [bad] + good[2:])) == 1
    assert L.s2o_cache_append(*([cache(Tq=0)] + good[1:])) == 0
    assert s2o.last_launch_count() == 0


def test_a_stride_that_reaches_no_row_says_nothing(L):
    """Of views with one token only the head stride counts, and stride_b of the append's
    never: such calls come past the views (to the refusal of too many heads)."""
    r, M = s2o.make_rotary(128), 1 << 30
    for T, odd in ((1, dict(b=3, t=1)), (1, dict(b=-1)), (2, dict(b=7)), (2, dict(b=1, t=1)), (1, dict(h=4))):
        c = cache(Hq=4096, Hkv=64, Tq=T)
        a = [view(i * M, **{**dict(t=1 << 20), **odd}) for i in range(1, 5)]
        got = L.s2o_cache_append(c, r, a[0], a[1], a[2], None, GOOD, GOOD, GOOD, ctypes.c_void_p(5 * M),
                                 ctypes.c_void_p(6 * M), a[3], None)
        assert got == (2 if "h" not in odd and odd.get("t", 8) % 8 * (T - 1) == 0 else 1), (T, odd)


def test_rotary_refusals(L):
    r = s2o.make_rotary(128)
    good = [r, 0, 1, 4, 2, 1, view(), view(), GOOD, view(), view(), 0, None]
    for i in (0, 6, 7, 8, 9, 10):
        assert L.s2o_rotary(*(good[:i] + [None] + good[i + 1:])) == 1, i
    for i, value in ((1, 2), (2, -1), (3, -1), (4, -1), (5, -1)):
        assert L.s2o_rotary(*(good[:i] + [value] + good[i + 1:])) == 1, i
    for i in (6, 7, 9, 10):
        assert L.s2o_rotary(*(good[:i] + [view(b=12)] + good[i + 1:])) == 1, i
    for i in (9, 10):  # an output whose rows fall on one another; an input may be broadcast
        assert L.s2o_rotary(*(good[:i] + [view(t=0)] + good[i + 1:])) == 1, i
    assert L.s2o_rotary(*(good[:4] + [5000] + good[5:])) == 2
    assert L.s2o_rotary(*(good[:3] + [0] + good[4:])) == 0  # nothing to turn
    assert s2o.last_launch_count() == 0


def test_binding_refuses_tensors_the_call_was_not_made_for():
    c, r = cache(), s2o.make_rotary(128)
    q, k = torch.zeros(3, 8, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    kc, vc = s2o.alloc_cache(c, "cpu")
    table, qs, kl = (torch.zeros(s, dtype=torch.int32) for s in ((2, 4), (3,), (2,)))
    bad = [dict(k=k.half()), dict(k=k[:2]), dict(q=q[:, :4]), dict(v=k.transpose(1, 2)), dict(k_cache=kc[:5]),
           dict(v_cache=vc.transpose(1, 2)), dict(page_table=table.long()), dict(q_start=qs[:2]),
           dict(kv_len=kl.float()), dict(positions=torch.zeros(2, 3, dtype=torch.int32)),
           dict(rotary=None, positions=torch.zeros(1, 3, dtype=torch.int32)), dict(q=None, q_out=q), dict()]
    for change in bad:  # the last one: right in all but the device
        a = dict(q=q, k=k, v=k, k_cache=kc, v_cache=vc, page_table=table, q_start=qs, kv_len=kl, rotary=r)
        a.update(change)
        with pytest.raises(s2o.S2OError) as e:
            s2o.cache_append(c, **a)
        assert e.value.code == 1
    pre = torch.zeros(2, dtype=torch.int32)
    for change in (dict(q=q.float()), dict(q=q.transpose(0, 1)), dict(prefix_pages=None), dict(prefix_pages=pre[:1]),
                   dict(O=q.float()), dict(lse=torch.zeros(3, 7)), dict()):
        a = dict(q=q, k_cache=kc, v_cache=vc, page_table=table, q_start=qs, kv_len=kl, prefix_pages=pre, O=q,
                 lse=torch.zeros(3, 8), workspace=torch.zeros(8))
        a.update(change)
        with pytest.raises(s2o.S2OError) as e:
            s2o.attention_paged(c, **a)
        assert e.value.code == 1
    x = torch.zeros(1, 3, 8, 128, dtype=torch.bfloat16)
    pos = torch.zeros(1, 1, 3, dtype=torch.int32)
    for change in (dict(q=x.float()), dict(q=x[0]), dict(k=x.half()), dict(k=x[:, :2]), dict(positions=pos[0]),
                   dict(positions=pos.long()), dict(positions=None), dict(q=x.transpose(2, 3)), dict(q_out=x[:, :, :4]),
                   dict(q=None, k=None), dict()):
        a = dict(q=x, k=x, positions=pos)
        a.update(change)
        with pytest.raises(s2o.S2OError) as e:
            s2o.rotary(r, **a)
        assert e.value.code == 1


def test_attention_without_a_workspace_refuses_host_tensors():
    c = cache()
    kc, vc = s2o.alloc_cache(c, "cpu")
    table, qs, kl, pre = (torch.zeros(s, dtype=torch.int32) for s in ((2, 4), (3,), (2,), (2,)))
    with pytest.raises(s2o.S2OError) as e:
        s2o.attention_paged(c, torch.zeros(3, 8, 128, dtype=torch.bfloat16), kc, vc, table, qs, kl, prefix_pages=pre)
    assert e.value.code == 1


def test_status_of_a_bad_cache(L):
    assert s2o.status_string(8) == "page, length or token range out of range"
    assert s2o.STATUS[8] == "S2O_ERR_BAD_CACHE"


VIEWS = r"""
#include "row_views.h"
using namespace s2o;
extern "C" {
int meet_self(int64_t p, const int64_t* s, const int64_t* n) {
  return rows_meet(RowView{reinterpret_cast<uint16_t*>(p), s[0], s[1], s[2]}, n[0], n[1], n[2]);
}
int meet_two(int64_t p, const int64_t* s, int64_t Hx, int64_t q, const int64_t* u, int64_t Hy, const int64_t* n) {
  return rows_meet(RowView{reinterpret_cast<uint16_t*>(p), s[0], s[1], s[2]}, Hx,
                   RowView{reinterpret_cast<uint16_t*>(q), u[0], u[1], u[2]}, Hy, n[0], n[1]);
}
}
"""


@pytest.fixture(scope="module")
def views(tmp_path_factory):
    d = tmp_path_factory.mktemp("views")
    (d / "v.cpp").write_text(VIEWS)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", build.CSRC, "-o", str(d / "v.so"),
                    str(d / "v.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "v.so"))
    arr = lambda x: (ctypes.c_int64 * 3)(*x)
    i64 = ctypes.c_int64
    return (lambda p, s, n: bool(lib.meet_self(i64(p), arr(s), arr(n))),
            lambda p, s, Hx, q, u, Hy, B, N: bool(lib.meet_two(i64(p), arr(s), i64(Hx), i64(q), arr(u), i64(Hy), arr((B, N, 0)))))


def elements(p, s, n):
    """Element ranges' first numbers of every row, from a byte address."""
    at = p // 2 + sum(np.arange(k).reshape([-1 if i == j else 1 for j in range(3)]) * st
                      for i, (k, st) in enumerate(zip(n, s)))
    return at.reshape(-1)


def some_strides(rng, n):
    """Nested in a random order, packed with room, or anything."""
    kind = rng.integers(3)
    if kind == 2:
        return [int(x) * 8 for x in rng.integers(-40, 200, 3)]
    s, reach = [0, 0, 0], 128 + 8 * int(rng.integers(0, 20)) * int(kind)
    for i in rng.permutation(3):
        s[i] = reach
        reach = reach * n[i] + 8 * int(rng.integers(0, 30)) * int(kind)
    return s


def test_rows_that_fall_on_one_another_are_seen(views):
    """Against a count of every element, on random views: of one view, and of two
    with the same strides (exact); of two with other strides no meeting is claimed
    that is none."""
    meet_self, meet_two = views
    rng = np.random.default_rng(7)
    base, hits = 1 << 30, [0, 0, 0, 0]
    for _ in range(6000):
        B, N, Hx, Hy = (int(x) for x in rng.integers(1, [4, 7, 6, 6]))
        s = some_strides(rng, (B, N, max(Hx, Hy) + 2))
        x = np.sort(elements(base, s, (B, N, Hx)))
        want = bool((np.diff(x) < 128).any())
        assert meet_self(base, s, (B, N, Hx)) == want, (s, B, N, Hx)
        hits[want] += 1
        q = base + 16 * int(rng.integers(-60, 200)) if rng.random() < .5 else base + 2 * s[2] * int(rng.integers(-2, 8))
        u = s if rng.random() < .7 else some_strides(rng, (B, N, Hy))
        y = elements(q, u, (B, N, Hy))
        want = bool((np.abs(x[:, None] - y[None]) < 128).any())
        got = meet_two(base, s, Hx, q, u, Hy, B, N)
        assert got == want if u is s else want or not got, (s, u, B, N, Hx, Hy, q - base)
        hits[2 + want] += 1
    assert min(hits) > 500, hits


def test_whole_buffers_in_another_order_are_seen(views):
    """Head-major rows over token-major ones, a window of them, strides that no memory has."""
    _, meet_two = views
    B, N, H = 2, 9, 5
    head, token = (H * N * 128, 128, N * 128), (N * H * 128, H * 128, 128)
    packed = (N * 9 * 128, 9 * 128, 128)
    assert meet_two(1 << 20, head, H, 1 << 20, token, H, B, N)
    assert meet_two(1 << 20, head, H, (1 << 20) + 2 * 128 * 7, token, H, B, N)
    assert not meet_two(1 << 20, head, H, (1 << 20) + 2 * 128 * B * N * H, token, H, B, N)
    assert meet_two(1 << 20, packed, 5, 1 << 20, head, H, B, N)
    assert not meet_two(1 << 20, packed, 5, (1 << 20) + 5 * 256, packed, 4, B, N)
    assert meet_two(1 << 20, packed, 5, (1 << 20) + 4 * 256, packed, 4, B, N)
    far = ((1 << 63) - 8, (1 << 62), -(1 << 63))
    assert meet_two(1 << 20, far, 5, 1 << 20, far, 5, B, N)


def test_outputs_in_the_way_are_refused(L):
    """An output on itself, on another output, or on an input it is not the place of."""
    r, M, X = s2o.make_rotary(128), 1 << 20, 1 << 30
    base = lambda **kw: {**dict(q=view(M), k=view(2 * M), qo=view(X), ko=view(X + M)), **kw}
    call = lambda a: L.s2o_rotary(r, 0, 1, 4, 2, 1, a["q"], a["k"], GOOD, a["qo"], a["ko"], 0, None)
    for bad in (dict(qo=view(X, t=64)), dict(qo=view(X, t=128, h=256)), dict(ko=view(X + 256)), dict(ko=view(X)),
                dict(qo=view(M, t=256)), dict(qo=view(M + 2 * 1024)), dict(ko=view(M + 256)), dict(qo=view(2 * M))):
        assert call(base(**bad)) == 1, list(bad)
    c = cache()
    good = dict(q=view(M), k=view(2 * M), v=view(3 * M), kc=ctypes.c_void_p(X), vc=ctypes.c_void_p(X + M), qo=view(M))
    for bad in (dict(qo=view(2 * M)), dict(qo=view(3 * M + 256)), dict(qo=view(M + 256)), dict(qo=view(M, t=128, h=384)),
                dict(qo=view(X, t=512, h=64)), dict(vc=ctypes.c_void_p(X + 256))):
        a = {**good, **bad}
        assert L.s2o_cache_append(c, r, a["q"], a["k"], a["v"], None, GOOD, GOOD, GOOD, a["kc"], a["vc"], a["qo"],
                                  None) == 1, list(bad)
    need = s2o.attention_paged_workspace_size(c)
    p = ctypes.c_void_p
    for O, f32 in ((X + 16, 0), (X + 3 * 8 * 256 - 16, 0), (X - 3 * 8 * 512 + 16, 1)):  # Q is 3 x 8 rows
        assert L.s2o_attention_paged(c, p(X), GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, p(O), f32, None, p(1 << 40), need,
                                     None) == 1
    assert s2o.last_launch_count() == 0
