"""Paged append and attention against their 64-bit forms, at the lengths, layouts and masks where
they can go wrong; captured graphs, other streams, reported errors and untouched rows."""
import math

import numpy as np
import pytest
import torch

from paged_ref import DT, HALF, U, Batch

pytestmark = pytest.mark.gpu

TYPES = [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")]
HEADS = [(16, 8, 128), (16, 2, 128), (4, 2, 64), (5, 1, 128), (14, 2, 64), (3, 3, 64), (12, 2, 128)]
# (new tokens, keys before): lengths around tile and page borders, empty ones among them
STEP = [(1, 0), (1, 14), (1, 15), (1, 16), (1, 62), (1, 63), (1, 64), (0, 0), (0, 40), (1, 127), (1, 700)]
CHUNKS = [(3, 0), (1, 33), (0, 5), (17, 60), (40, 0), (2, 255), (9, 119)]


def attend_close(b, got, ref=None):
    want, tol = ref or b.attend()
    got = got[:b.tokens].double().cpu()
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())
    # independent roundings add up as a root: far below the bound above
    rel = float((got - want).norm() / want.norm()) if float(want.norm()) else 0.0
    assert rel <= (4e-6 if b.act == "f32" else 1e-2), rel


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("nq,nkv,hd", HEADS)
def test_attend_steps(act, kv, nq, nkv, hd):
    b = Batch(STEP, nq, nkv, hd, 16, act, kv, seed=1)
    c = b.cache()
    attend_close(b, c.attend(b.q.cuda()))
    c.check()


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_attend_pages(act, kv, page):
    b = Batch([(1, 0), (1, 100), (1, 255), (1, 256), (1, 511)], 8, 2, 128, page, act, kv, seed=2)
    c = b.cache()
    attend_close(b, c.attend(b.q.cuda()))
    c.check()


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (16, 2, 128), (5, 1, 128), (7, 1, 64)])
def test_attend_chunks(act, kv, nq, nkv, hd):
    b = Batch(CHUNKS, nq, nkv, hd, 16, act, kv, seed=3)
    c = b.cache()
    ref = b.attend()
    attend_close(b, c.attend(b.q.cuda(), max_new=40), ref)
    attend_close(b, c.attend(b.q.cuda(), max_new=1), ref)   # a wrong hint costs speed only
    c.check()


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("prefix", [1, 16, 63, 64, 65, 300])
def test_attend_prefix(act, kv, prefix):
    # sequences without own keys see the prefix alone
    b = Batch([(1, 0), (1, 30), (0, 3), (1, 64), (2, 10)] + [(1, 3)] * 9, 8, 2, 64, 16, act, kv,
              prefix=prefix, pad=2, seed=prefix)
    c = b.cache()
    attend_close(b, c.attend(b.q.cuda(), max_new=2))
    c.check()


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("nq,nkv,hd", [(16, 2, 128), (4, 2, 64)])
def test_attend_prefix_and_chunks(act, kv, nq, nkv, hd):
    b = Batch([(30, 0), (1, 70), (45, 20)], nq, nkv, hd, 32, act, kv, prefix=130, seed=5)
    c = b.cache()
    attend_close(b, c.attend(b.q.cuda(), max_new=45))
    c.check()


def test_rows_without_a_key_are_zero():
    # kv_len 0 with one token: nothing to see; and with a prefix the prefix alone
    for act, kv in TYPES:
        for prefix in (0, 20):
            b = Batch([(1, 5), (1, 0)], 4, 2, 64, 16, act, kv, prefix=prefix, seed=7)
            b.len[1] = 0
            c = b.cache()
            got = c.attend(b.q.cuda())[1].double().cpu()
            if prefix == 0:
                assert (got == 0).all()
            else:
                k, v = b.keys(b.k, 1), b.keys(b.v, 1)
                for h in range(4):
                    p = torch.softmax(k[h // 2] @ b.q[1, h].double() / 8.0, 0)
                    want = p @ v[h // 2]
                    # 20 keys: a bf16 P and output round by 2^-8 of at most max |v| each
                    tol = 1e-5 if "f32" in (act, kv) and act == "f32" else 2 * HALF["bf16"] * float(v.abs().max())
                    assert (got[h] - want).abs().max() <= tol


@pytest.mark.parametrize("act,kv", TYPES)
def test_chunks_whose_first_tokens_see_nothing(act, kv):
    # kv_len below the new tokens: reported, the tokens before the first key get zeros (or the
    # prefix alone), the others what they see; with many rows per key and with few
    for prefix, new, length in [(0, 150, 40), (0, 9, 2), (33, 150, 0)]:
        b = Batch([(new, 0), (1, 70)], 8, 2, 64, 16, act, kv, prefix=prefix, seed=89)
        b.len[0] = length
        c = b.cache()
        got = c.attend(b.q.cuda(), max_new=new).double().cpu()
        assert torch.isfinite(got).all()
        if prefix == 0:
            assert (got[:new - length] == 0).all()
        k, v = b.keys(b.k, 0), b.keys(b.v, 0)
        for i in (0, new // 2, new - 1):
            n = prefix + max(0, length - new + i + 1)
            for h in (0, 5):
                p = torch.softmax(k[h // 4, :n] @ b.q[i, h].double() / 8.0, 0)
                want = p @ v[h // 4, :n]
                # up to 73 keys: f32 sums (1e-5 of values below 5), or bf16 weights and output
                tol = 1e-4 if act == "f32" else 2 * HALF["bf16"] * float(v.abs().max())
                assert n == 0 or (got[i, h] - want).abs().max() <= tol
        with pytest.raises(RuntimeError, match="BAD_LENGTH"):
            c.check()


@pytest.mark.parametrize("act,kv", TYPES)
def test_large_scores_and_ties(act, kv):
    # one key far above the rest, equal keys, and large values: the softmax's reference moves
    b = Batch([(1, 300), (1, 90)], 4, 2, 64, 16, act, kv, seed=9)
    at, slot = b.table[0, 250 // 16], 250 % 16
    b.k[at, :, slot] = (b.q[0, 0].double() * 8).to(DT[kv])
    b.k[b.table[1, 0], :, :8] = 0.0
    b.v[b.table[1, 1]] *= 1000
    c = b.cache()
    attend_close(b, c.attend(b.q.cuda()))


@pytest.mark.parametrize("act,kv", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_long_split_sequences(act, kv):
    # one long and many short sequences: items split over many CTAs, and the same bits again
    b = Batch([(1, 3000)] + [(1, i) for i in range(40)], 8, 1, 64, 64, act, kv, seed=11)
    c = b.cache()
    q = b.q.cuda()
    got = c.attend(q)
    attend_close(b, got)
    for _ in range(3):
        assert torch.equal(c.attend(q), got)


@pytest.mark.parametrize("act,kv", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("nq,nkv,hd,page", [(8, 2, 64, 16), (4, 2, 128, 64), (6, 2, 128, 32), (1, 1, 64, 256)])
def test_long_chunks(act, kv, nq, nkv, hd, page):
    # several row tiles per sequence, diagonals inside and across key tiles, short ones beside them
    b = Batch([(300, 10), (129, 0), (1, 500), (64, 200), (0, 30), (2, 127)], nq, nkv, hd, page, act, kv,
              seed=61)
    c = b.cache()
    got = c.attend(b.q.cuda(), max_new=300)
    attend_close(b, got)
    assert torch.equal(c.attend(b.q.cuda(), max_new=300), got)
    c.check()


@pytest.mark.parametrize("act,kv", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("nq,nkv,hd", [(16, 2, 64), (2, 1, 128)])
def test_prefix_of_a_large_batch(act, kv, nq, nkv, hd):
    # many row tiles share the prefix; most of its items are split over several CTAs
    b = Batch([(1, i % 40) for i in range(100)] + [(0, 3), (3, 0)], nq, nkv, hd, 16, act, kv, prefix=1037,
              pad=1, seed=67)
    c = b.cache()
    got = c.attend(b.q.cuda())
    attend_close(b, got)
    for _ in range(2):
        assert torch.equal(c.attend(b.q.cuda())[:b.tokens], got[:b.tokens])
    c.check()


def test_chunk_of_one_long_sequence():
    # few items, each split over many CTAs and joined by a kernel of its own
    for act in ("f32", "bf16"):
        b = Batch([(40, 2500)], 2, 1, 128, 64, act, "bf16", seed=71)
        c = b.cache()
        attend_close(b, c.attend(b.q.cuda(), max_new=40))
        c.check()


@pytest.mark.parametrize("kv,prefix,tokens", [("bf16", 8192, 512), ("bf16", 3000, 40), ("f32", 8192, 64)])
def test_f32_results_at_long_prefixes(kv, prefix, tokens):
    """The tensor cores add with rounding towards zero, up to 2^-23 of the sum per product: 48 of
    them at most run into one accumulator (5.7e-6), whatever the length."""
    nq, nkv, hd, page = 64, 8, 128, 64
    from sequence_decode_step_gb300 import PagedKV
    g = torch.Generator(device="cuda").manual_seed(5)
    n = -(-prefix // page)
    k = torch.randn(n + 1, nkv, page, hd, generator=g, device="cuda").to(DT[kv])
    v = torch.randn(n + 1, nkv, page, hd, generator=g, device="cuda").to(DT[kv])
    q = torch.randn(tokens, nq, hd, generator=g, device="cuda") * 1.5
    i32 = {"device": "cuda", "dtype": torch.int32}
    c = PagedKV(k, v, torch.full((tokens, 1), n, **i32), torch.ones(tokens, **i32),
                torch.arange(tokens + 1, **i32), prefix_pages=torch.arange(n, **i32), prefix_len=prefix)
    got = c.attend(q)[-2:].double()
    # the prefix, then the one key of their own: the first of the last page, for all of them
    kk, vv = (torch.cat([t[:n].permute(1, 0, 2, 3).reshape(nkv, -1, hd)[:, :prefix], t[n, :, :1]], 1).double()
              for t in (k, v))
    s = torch.einsum("thgd,hkd->thgk", q[-2:].double().view(2, nkv, -1, hd), kk) / math.sqrt(hd)
    want = torch.einsum("thgk,hkd->thgd", torch.softmax(s, -1), vv).reshape(2, nq, hd)
    assert float((got - want).norm() / want.norm()) <= 6e-6
    c.check()


@pytest.mark.parametrize("kv,hd", [("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("new", [(5,), (6, 4)])
def test_few_tokens_behind_a_long_prefix_beside_other_work(kv, hd, new):
    """Both launches of a call take tensor-core tiles whose O moves to records, with so few rows that the
    joining kernel between them starts early; another stream's products make CTAs start late. The second
    launch may then run beside the first: the same bits every time, and the right ones."""
    from sequence_decode_step_gb300 import PagedKV
    nq, nkv, page, prefix, own = 64, 8, 64, 20000, 16500
    g = torch.Generator(device="cuda").manual_seed(11)
    npre, per = -(-prefix // page), -(-own // page)
    k, v = (torch.randn(npre + len(new) * per, nkv, page, hd, generator=g, device="cuda").to(DT[kv])
            for _ in range(2))
    i32 = {"device": "cuda", "dtype": torch.int32}
    n = sum(new)
    q = torch.randn(n, nq, hd, generator=g, device="cuda") * 1.5
    table = npre + torch.arange(len(new) * per, **i32).view(len(new), per)
    lens = [own - 37 * b for b in range(len(new))]
    c = PagedKV(k, v, table, torch.tensor(lens, **i32), torch.tensor(np.cumsum([0, *new]), **i32),
                prefix_pages=torch.arange(npre, **i32), prefix_len=prefix)
    first = c.attend(q, max_new=max(new))
    t = 0
    for b, m in enumerate(new):
        kk, vv = (torch.cat([x[:npre].permute(1, 0, 2, 3).reshape(nkv, -1, hd)[:, :prefix],
                             x[table[b].long()].permute(1, 0, 2, 3).reshape(nkv, -1, hd)[:, :lens[b]]], 1).double()
                  for x in (k, v))
        s = torch.einsum("thgd,hkd->thgk", q[t:t + m].double().view(m, nkv, -1, hd), kk) / math.sqrt(hd)
        see = torch.arange(kk.shape[1], device="cuda")[None] < (
            prefix + lens[b] - m + 1 + torch.arange(m, device="cuda")[:, None])
        p = torch.softmax(s.masked_fill(~see[:, None, None], -math.inf), -1)
        want = torch.einsum("thgk,hkd->thgd", p, vv).reshape(m, nq, hd)
        # 48 products of at most 2^-23 each run into one accumulator (5.7e-6 of the values, at most)
        assert float((first[t:t + m].double() - want).norm() / want.norm()) <= 6e-6
        t += m
    side = torch.cuda.Stream()
    x = torch.randn(1500, 1500, device="cuda")
    torch.cuda.synchronize()
    for i in range(30):
        with torch.cuda.stream(side):
            for _ in range(1 + i % 4):
                x @ x
        got = [c.attend(q, max_new=max(new)) for _ in range(3)]
        assert all(torch.equal(y, first) for y in got)
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("nq,nkv,hd,page,prefix", [
    (8, 2, 64, 16, 0), (16, 2, 128, 64, 130), (5, 1, 128, 32, 0), (7, 1, 64, 256, 65), (3, 3, 128, 128, 1100)])
def test_f32_pages_of_wide_tables(act, nq, nkv, hd, page, prefix):
    # the longest sequence that the table could hold decides the kernel: tiles of 128 rows here, with
    # ends inside tiles, diagonals, a sequence without tokens and items split over several CTAs
    b = Batch([(150, 10), (129, 0), (1, 700), (64, 200), (0, 30), (2, 127), (40, 1100)], nq, nkv, hd, page,
              act, "f32", prefix=prefix, pad=2, seed=97, extra_cols=32768 // page)
    c = b.cache()
    out = torch.full((b.rows, nq, hd), 7.0, dtype=DT[act], device="cuda")
    got = c.attend(b.q.cuda(), max_new=150, out=out)
    attend_close(b, got)
    assert (got[b.tokens:] == 7.0).all()
    for _ in range(2):
        assert torch.equal(c.attend(b.q.cuda(), max_new=150)[:b.tokens], got[:b.tokens])
    c.check()


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("nq,nkv,hd", [(14, 2, 64), (16, 2, 128)])
def test_two_tokens_over_many_keys(act, kv, nq, nkv, hd):
    # 14 and 16 rows per key, split over all CTAs: the most records that the smallest workspace holds
    for seqs, prefix in (([(1, 20), (1, 300)], 9001), ([(2, 9000)], 0)):
        b = Batch(seqs, nq, nkv, hd, 64, act, kv, prefix=prefix, seed=107)
        c = b.cache()
        attend_close(b, c.attend(b.q.cuda(), max_new=2))
        c.check()


@pytest.mark.parametrize("act,kv", TYPES)
def test_many_short_chunks_in_wide_tables(act, kv):
    # several items per CTA, most of which fill one row tile of two: the other one's warps run ahead
    b = Batch([(1 + 13 * i % 41, 0) for i in range(60)] + [(150, 3)], 16, 8, 64, 64, act, kv, seed=103,
              extra_cols=512)
    c = b.cache()
    q = b.q.cuda()
    got = c.attend(q, max_new=150)
    attend_close(b, got)
    for _ in range(20):
        assert torch.equal(c.attend(q, max_new=150), got)
    c.check()


@pytest.mark.parametrize("act,kv,nq", [("bf16", "bf16", 32), ("f32", "bf16", 32), ("f32", "f32", 16), ("f32", "f32", 64),
                                       ("bf16", "f32", 32)])
@pytest.mark.parametrize("prefix", [0, 1386])
def test_every_tile_is_read_before_its_stage_is_filled_again(act, kv, nq, prefix):
    """Keys of zero weigh all rows alike, and a value row is the unit vector of its 32-key block (mod
    128): column d of the output counts the keys of such blocks, exactly in f32. Over and over, since a
    copy that overtakes a read is rare."""
    from sequence_decode_step_gb300 import PagedKV
    nkv, hd, page, n = 8, 128, 64, 161
    r = np.random.RandomState(3)
    lens = r.randint(1, 4096, size=n)
    pages = -(-lens // page)
    total, npre = int(pages.sum()), -(-prefix // page)
    perm, table, at = r.permutation(total), np.zeros((n, int(pages.max())), np.int32), 0
    block = np.zeros((total, page), np.int64)
    for b in range(n):
        ids = perm[at:at + pages[b]]
        table[b, :pages[b]] = ids
        at += pages[b]
        block[ids] = np.arange(pages[b] * page).reshape(-1, page) // 32
    k = torch.zeros(total + npre + 1, nkv, page, hd, device="cuda", dtype=DT[kv])
    v = torch.zeros_like(k)
    v[:total] = torch.nn.functional.one_hot(torch.from_numpy(block).cuda() % 128, 128).to(DT[kv])[:, None]
    i32 = {"device": "cuda", "dtype": torch.int32}
    c = PagedKV(k, v, torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(),
                torch.arange(n + 1, **i32), prefix_len=prefix,
                prefix_pages=torch.arange(total, total + npre, **i32) if prefix else None)
    q = torch.randn(n, nq, hd, device="cuda").to(DT[act])
    length = torch.from_numpy(lens).cuda()
    count = (length[:, None] - 32 * torch.arange(128, device="cuda")[None]).clamp(0, 32).double()
    want = (count / (length[:, None] + prefix))[:, None]
    for _ in range(25):
        # products of 0 and 1 and their sums are exact; a reciprocal, a product and the output's rounding
        # follow, and one key more or less changes a count by 1/32 of it at least
        assert ((c.attend(q).double() - want).abs() <= want * (HALF[act] + 4 * U)).all()
    c.check()


def test_f32_pages_of_wide_tables_bad_entries():
    # a page outside the pool is read as page 0, tokens before the first key get zeros, both reported
    b = Batch([(150, 300), (100, 0)], 8, 2, 64, 16, "f32", "f32", seed=101, extra_cols=2048)
    b.table[0, 3] = b.n_pages
    b.table[0, 5] = -1
    b.k[0] = b.v[0] = 0.5
    b.len[1] = 30
    c = b.cache()
    got = c.attend(b.q.cuda(), max_new=150)[:b.tokens]
    assert torch.isfinite(got).all() and (got[150:220] == 0).all() and (got[220:] != 0).any(-1).all()
    with pytest.raises(RuntimeError, match="BAD_PAGE.*BAD_LENGTH|BAD_LENGTH.*BAD_PAGE"):
        c.check()


def test_padding_rows_are_left_and_strides():
    for act, kv in TYPES:
        b = Batch([(2, 9), (1, 40)], 4, 2, 64, 16, act, kv, pad=3, seed=13)
        c = b.cache()
        wide = torch.full((b.rows, 4 * 64 + 64), math.nan, dtype=DT[act], device="cuda")
        wide[:, :256] = b.q.cuda().reshape(b.rows, 256)
        out = torch.full((b.rows, 4, 64), 7.0, dtype=DT[act], device="cuda")
        got = c.attend(wide[:, :256], max_new=2, out=out)
        attend_close(b, got)
        assert (got[b.tokens:] == 7.0).all()
        qkv = torch.full((b.rows, 8 * 64 + 8), math.nan, dtype=DT[act], device="cuda")
        qkv[:, :512] = b.qkv.cuda()
        out = torch.full((b.rows, 4, 64), 7.0, dtype=DT[act], device="cuda")
        got = c.append(qkv[:, :512], 4, out=out)
        assert (got[b.tokens:] == 7.0).all()
        check_append(b, got, {})


# ------------------------------------------------------------------------------- append
# Roundings of an f32 rotation: the turn's fraction (four of 2^-25 turns, 7.5e-7 rad), sincospif
# and the two products (about 6 U), the norm (rsqrtf 2 ulp, its sum of at most 18 adds, two
# products): below 2e-6 of |x_j| + |x_{j+hd/2}|.
ROT = 2e-6


def check_append(b, got, kw):
    q, k, v, qs, ks = b.append(**kw)
    n = b.tokens
    tol = ROT * qs + HALF[b.act] * (b.act != "f32") * q.abs()
    assert ((got[:n].double().cpu() - q).abs() <= tol).all()
    at, slot = b.slots()
    at_t, slot_t = torch.from_numpy(at), torch.from_numpy(slot)
    kd, vd = b.kd.cpu(), b.vd.cpu()
    kk, vv = kd[at_t, :, slot_t].double(), vd[at_t, :, slot_t].double()
    tol = ROT * ks + HALF[b.kv] * (b.kv != "f32") * k.abs()
    assert ((kk - k).abs() <= tol).all()
    assert torch.equal(vv, v.to(DT[b.kv]).double())
    # every other slot is left as it was
    old_k, old_v = b.k.clone(), b.v.clone()
    old_k[at_t, :, slot_t] = kd[at_t, :, slot_t]
    old_v[at_t, :, slot_t] = vd[at_t, :, slot_t]
    bits = torch.int16 if b.kv == "bf16" else torch.int32
    assert torch.equal(old_k.view(bits), kd.view(bits))
    assert torch.equal(old_v.view(bits), vd.view(bits))


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("nq,nkv,hd", HEADS)
@pytest.mark.parametrize("norm", [False, True])
def test_append(act, kv, nq, nkv, hd, norm):
    b = Batch(CHUNKS + [(1, 0), (1, 15), (1, 16)], nq, nkv, hd, 16, act, kv, seed=17)
    c = b.cache()
    kw = {}
    if norm:
        g = torch.Generator().manual_seed(3)
        kw = {"q_norm": (1 + 0.1 * torch.randn(hd, generator=g)).to(torch.bfloat16),
              "k_norm": (1 + 0.1 * torch.randn(hd, generator=g)).to(torch.bfloat16), "eps": 1e-6}
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    check_append(b, c.append(b.qkv.cuda(), nq, **dev), kw)
    c.check()


@pytest.mark.parametrize("act,kv", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("hd,sections", [(128, (16, 24, 24)), (64, (8, 0, 24)), (64, (0, 0, 32)),
                                         (128, (64, 0, 0))])
def test_append_three_axes(act, kv, hd, sections):
    b = Batch([(37, 3), (1, 80), (5, 0)], 4, 2, hd, 32, act, kv, prefix=10, seed=19)
    c = b.cache()
    r = np.random.default_rng(1)
    pos = torch.from_numpy(r.integers(0, 1 << 20, (b.rows, 3)).astype(np.int32))
    got = c.append(b.qkv.cuda(), 4, positions=pos.cuda(), sections=sections, rope_theta=1e6)
    check_append(b, got, {"positions": pos, "sections": sections})


def test_append_far_and_negative_positions():
    b = Batch([(64, 0)], 2, 1, 128, 64, "f32", "f32", seed=23)
    c = b.cache()
    pos = torch.tensor([0, 1, -1, 65535, 65536, 131071, -65537, (1 << 24) - 1, 1 << 24, -(1 << 24)] * 6 +
                       [5, 6, 7, 8], dtype=torch.int32)
    got = c.append(b.qkv.cuda(), 2, positions=pos.cuda(), rope_theta=1e4)
    check_append(b, got, {"positions": pos, "theta": 1e4})


@pytest.mark.parametrize("theta", [1.0, 5e8, 3e38])
def test_append_at_the_ends_of_theta(theta):
    # one frequency for all pairs, and frequencies down to subnormal ones
    b = Batch([(6, 0)], 2, 1, 64, 64, "f32", "f32", seed=139)
    c = b.cache()
    pos = torch.tensor([0, 1, 65537, 999999, (1 << 24) - 1, -(1 << 24)], dtype=torch.int32)
    theta = float(np.float32(theta))
    check_append(b, c.append(b.qkv.cuda(), 2, positions=pos.cuda(), rope_theta=theta), {"positions": pos, "theta": theta})


def test_prefix_shifts_the_default_positions():
    b = Batch([(3, 4), (1, 0)], 4, 2, 64, 16, "f32", "bf16", prefix=77, seed=29)
    c = b.cache()
    check_append(b, c.append(b.qkv.cuda(), 4), {})


def test_many_sequences():
    b = Batch([(1, i % 7) for i in range(700)], 2, 1, 64, 16, "f32", "bf16", seed=31)
    c = b.cache()
    check_append(b, c.append(b.qkv.cuda(), 2), {})
    b.k, b.v = b.kd.cpu(), b.vd.cpu()
    attend_close(b, c.attend(b.q.cuda()))


# ------------------------------------------------------------------------------- together
@pytest.mark.parametrize("act,kv", TYPES)
def test_append_then_attend_as_a_server_does(act, kv):
    """A prompt in two chunks, then steps, against attention over the exact rotated keys."""
    b = Batch([(0, 0), (0, 0)], 8, 2, 64, 16, act, kv, prefix=40, seed=37, extra_cols=12)
    total = [50, 21]
    r = np.random.default_rng(5)
    # pages for the whole conversation
    need = [-(-t // 16) for t in total]
    pool = torch.full((sum(need) + len(b.pre) + 3, 2, 16, 64), math.nan, dtype=DT[kv])
    pre = np.arange(sum(need), sum(need) + len(b.pre))
    for i, p in enumerate(b.pre):
        pool[pre[i]] = b.k[p]
    b.n_pages, b.pre, b.k, b.v = pool.shape[0], pre, pool, pool.clone()
    order = r.permutation(sum(need))
    b.table[0, :need[0]], b.table[1, :need[1]] = order[:need[0]], order[need[0]:]
    b.new, b.len, b.tokens, b.rows = np.array([1, 1]), np.array([1, 1]), 2, 2
    c = b.cache()
    done = [0, 0]
    for step in [(30, 5), (13, 9), (1, 1), (1, 1), (5, 0), (0, 5)]:
        b.new = np.array(step)
        done = [done[0] + step[0], done[1] + step[1]]
        b.len, b.tokens = np.array(done), sum(step)
        b.rows, b.start = b.tokens, np.concatenate([[0], np.cumsum(step)])
        b.len_d.copy_(torch.from_numpy(b.len.astype(np.int32)))
        b.start_d.copy_(torch.from_numpy(b.start.astype(np.int32)))
        b.qkv = torch.from_numpy(r.standard_normal((b.tokens, 12 * 64))).to(DT[act])
        q = c.append(b.qkv.cuda(), 8, positions=None)
        check_append(b, q, {})
        got = c.attend(q, max_new=max(step))
        b.k, b.v, b.q = b.kd.cpu(), b.vd.cpu(), q.cpu()
        attend_close(b, got)
    c.check()


def test_captured_graph_replays_with_new_lengths():
    b = Batch([(1, 200), (1, 17), (1, 90)], 8, 2, 128, 16, "f32", "bf16", prefix=33, seed=41)
    c = b.cache()
    q, qkv = b.q.cuda(), b.qkv.cuda()
    out = torch.zeros(b.rows, 8, 128, device="cuda")
    rot = torch.zeros_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.append(qkv, 8, out=rot)
        c.attend(q, out=out)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(qkv, 8, out=rot)
        c.attend(q, out=out)
    for lens in ([201, 18, 91], [60, 3, 16], [1, 1, 1]):
        b.len = np.array(lens)
        b.len_d.copy_(torch.from_numpy(b.len.astype(np.int32)))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        b.k, b.v = b.kd.cpu(), b.vd.cpu()
        attend_close(b, out)
    c.check()


@pytest.mark.parametrize("act,kv", TYPES)
def test_captured_chunks_replay_with_new_lengths_and_starts(act, kv):
    # chunks behind a prefix on tensor-core tiles (four launches), fewer tokens than captured in some replays
    b = Batch([(40, 200), (1, 17), (23, 90)], 16, 2, 64, 16, act, kv, prefix=333, pad=3, seed=163, extra_cols=2048)
    c = b.cache()
    q, qkv = b.q.cuda(), b.qkv.cuda()
    out, rot = torch.zeros_like(q), torch.zeros_like(q)
    c.reserve(b.rows, 16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(qkv, 16, out=rot)
        c.attend(q, max_new=40, out=out)
    for new, lens in (([40, 1, 23], [240, 18, 113]), ([2, 30, 0], [9, 30, 5]), ([0, 0, 1], [0, 16, 113]),
                      ([33, 20, 11], [33, 20, 11])):
        b.new, b.len, b.tokens = np.array(new), np.array(lens), sum(new)
        b.start = np.concatenate([[0], np.cumsum(new)])
        b.len_d.copy_(torch.from_numpy(b.len.astype(np.int32)))
        b.start_d.copy_(torch.from_numpy(b.start.astype(np.int32)))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        b.k, b.v = b.kd.cpu(), b.vd.cpu()
        attend_close(b, out)
        assert (out[b.tokens:] == 7.0).all()
    c.check()


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("nq,new,cols", [(4, 1, 1), (16, 1, 1), (16, 30, 2048)])
def test_pools_past_2_31_elements(act, kv, nq, new, cols):
    """The batch's pages at the end of a pool of 2.2e9 elements, on every kernel; what lies at the same
    place modulo 2^32 bytes or 2^31 elements is other data."""
    from sequence_decode_step_gb300 import PagedKV
    b = Batch([(new, 700), (1, 33), (new, 0)], nq, 2, 128, 256, act, kv, prefix=600, seed=167, extra_cols=cols)
    n = 33600
    pools = [torch.empty(n, 2, 256, 128, dtype=DT[kv], device="cuda") for _ in range(2)]
    assert pools[0].numel() > (1 << 31) + (1 << 24)
    for big, small in zip(pools, (b.k, b.v)):
        big[-b.n_pages:] = small.cuda()
        big[:b.n_pages + 1024] = 3.0
    i32 = {"device": "cuda", "dtype": torch.int32}
    table = torch.from_numpy(np.where(b.table < b.n_pages, b.table + n - b.n_pages, 1 << 30).astype(np.int32)).cuda()
    c = PagedKV(*pools, table, torch.from_numpy(b.len.astype(np.int32)).cuda(),
                torch.from_numpy(b.start.astype(np.int32)).cuda(),
                prefix_pages=torch.from_numpy(b.pre + n - b.n_pages).to(**i32), prefix_len=600)
    attend_close(b, c.attend(b.q.cuda(), max_new=new))
    got = c.append(b.qkv.cuda(), nq)
    b.kd, b.vd = (p[-b.n_pages:].clone() for p in pools)
    check_append(b, got, {})
    assert all((p[:b.n_pages + 1024] == 3.0).all() for p in pools)
    c.check()
    del c, pools
    torch.cuda.empty_cache()


def test_capture_needs_its_workspace_and_keeps_it():
    b = Batch([(1, 200), (1, 17)], 4, 2, 64, 16, "f32", "bf16", seed=73)
    c = b.cache()
    q, out = b.q.cuda(), torch.zeros(2, 4, 64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="reserve"):
        with torch.cuda.graph(g):
            c.attend(q, out=out)
    torch.cuda.synchronize()
    c.reserve(2, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(q, out=out)
    c.reserve(4096, 4)                            # a larger one must not take the graph's away
    filler = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    g.replay()
    attend_close(b, out)
    attend_close(b, c.attend(q))
    del filler


def test_layers_share_a_workspace():
    a = Batch([(1, 300), (1, 5)], 4, 2, 64, 16, "f32", "bf16", prefix=20, seed=79)
    b = Batch([(1, 300), (1, 5)], 4, 2, 64, 16, "f32", "bf16", prefix=20, seed=83)
    ca = a.cache()
    cb = b.cache(workspace=ca.workspace)
    ca.reserve(2, 4)
    q = [a.q.cuda(), b.q.cuda()]
    got = [(ca.attend(q[0]), cb.attend(q[1])) for _ in range(3)]
    for x, y in got:
        attend_close(a, x)
        attend_close(b, y)
    assert ca.workspace is cb.workspace and len(ca.workspace._kept) == 1
    for n in range(3, 400):                       # growing batches do not pile up workspaces
        ca.reserve(n, 4)
    assert len(ca.workspace._kept) <= 4


def test_other_streams():
    b = Batch([(1, 500), (1, 3)], 8, 2, 128, 16, "bf16", "bf16", seed=43)
    c = b.cache()
    q = b.q.cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = c.attend(q)
    s.synchronize()
    attend_close(b, got)


@pytest.mark.parametrize("act,kv", TYPES)
def test_two_streams_at_once(act, kv):
    # a batch of steps behind a prefix on one stream, chunks on another, a workspace each: the same bits as alone
    a = Batch([(1, 300 + 7 * i) for i in range(20)], 8, 2, 64, 16, act, kv, prefix=500, seed=151)
    b = Batch([(60, 200), (1, 900), (33, 0)], 16, 2, 64, 16, act, kv, seed=157, extra_cols=2048)
    ca, cb = a.cache(), b.cache()
    qa, qb = a.q.cuda(), b.q.cuda()
    alone = [ca.attend(qa), cb.attend(qb, max_new=60)]
    attend_close(a, alone[0])
    attend_close(b, alone[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            got[0].append(ca.attend(qa))
        with torch.cuda.stream(streams[1]):
            got[1].append(cb.attend(qb, max_new=60))
    torch.cuda.synchronize()
    for x, y in zip(got, alone):
        assert all(torch.equal(t, y) for t in x)
    ca.check()
    cb.check()


def test_scratch_outlives_its_cache_on_other_streams():
    """Made on one stream, used on another, dropped while that one is still busy: nobody gets the memory."""
    import gc
    b = Batch([(1, 500), (1, 3)], 8, 2, 128, 16, "bf16", "bf16", prefix=40, seed=43)
    c = b.cache()
    c.reserve(2, 8)
    q = b.q.cuda()
    out = torch.zeros_like(q)
    mine = [c.workspace.ptr, c.status.data_ptr()]
    size = c.workspace.bytes
    gc.collect()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(1 << 30)               # half a second
        c.attend(q, out=out)
    del c
    other = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
    words = [torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(4096)]
    busy = not s.query()
    taken = {t.data_ptr() for t in other + words} & set(mine)
    s.synchronize()
    assert busy and not taken
    attend_close(b, out)


# ------------------------------------------------------------------------------- reported errors
def test_bad_pages_and_lengths_are_reported():
    b = Batch([(1, 20), (1, 20)], 4, 2, 64, 16, "f32", "bf16", seed=47)
    good, tol = b.attend()
    b.table[0, 0] = b.n_pages
    c = b.cache()
    got = c.attend(b.q.cuda()).double().cpu()
    assert ((got[1] - good[1]).abs() <= tol[1]).all()          # the other sequence is not affected
    with pytest.raises(RuntimeError, match="BAD_PAGE"):
        c.check()
    c.status.zero_()
    b.table_d[0, 1] = -5                                       # the new token's own page
    before = b.kd.clone()
    c.append(b.qkv.cuda(), 4)
    with pytest.raises(RuntimeError, match="BAD_PAGE"):
        c.check()
    at, slot = b.table[1, 1], 20 % 16                          # only sequence 1 was written
    before[at, :, slot] = b.kd[at, :, slot]
    assert torch.equal(before.view(torch.int16), b.kd.view(torch.int16))
    c.status.zero_()
    b.len_d[1] = 10000                                         # past the table
    c.append(b.qkv.cuda(), 4)
    with pytest.raises(RuntimeError, match="BAD_LENGTH"):
        c.check()
    c.status.zero_()
    c.attend(b.q.cuda())
    with pytest.raises(RuntimeError, match="BAD_LENGTH"):
        c.check()


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("nq,cols", [(4, 1), (16, 2048)])
def test_sequences_past_the_rows_of_a_call(act, kv, nq, cols):
    # a q_start that goes on behind the call's rows (a graph of fewer tokens): the rows that are there keep
    # their positions, see the keys that they see otherwise, and the rest is reported by both calls
    b = Batch([(3, 10), (40, 20), (2, 7)], nq, 2, 64, 16, act, kv, seed=127, extra_cols=cols)
    want, tol = b.attend()
    n = 30
    c = b.cache()
    got = c.attend(b.q.cuda()[:n], max_new=40).double().cpu()
    assert ((got - want[:n]).abs() <= tol[:n]).all()
    with pytest.raises(RuntimeError, match="BAD_LENGTH"):
        c.check()
    d, e = b.cache(), b.cache()
    qkv = torch.randn(b.rows, (nq + 4) * 64, device="cuda").to(DT[act])
    short, whole = d.append(qkv[:n], nq), e.append(qkv, nq)
    assert torch.equal(short, whole[:n])
    with pytest.raises(RuntimeError, match="BAD_LENGTH"):
        d.check()
    e.check()


def test_starts_that_decrease_are_reported():
    b = Batch([(2, 10), (3, 20)], 4, 2, 64, 16, "f32", "bf16", seed=131)
    for start in ([0, 3, 2], [-1, 2, 5]):
        for call in ("append", "attend"):
            c = b.cache()
            b.start_d.copy_(torch.tensor(start, dtype=torch.int32))
            c.append(b.qkv.cuda(), 4) if call == "append" else c.attend(b.q.cuda(), max_new=3)
            with pytest.raises(RuntimeError, match="BAD_LENGTH"):
                c.check()


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("nq,cols", [(4, 1), (16, 2048)])
def test_starts_that_decrease_behind_a_prefix(act, kv, nq, cols):
    # rows that the prefix's launch did not take have no records to join: the call does nothing, is reported
    # and its workspace serves the next one
    b = Batch([(5, 10), (3, 20), (8, 0)], nq, 2, 64, 16, act, kv, prefix=3000, seed=149, extra_cols=cols)
    c = b.cache()
    q = b.q.cuda()
    for start in ([5, 0, 3, 3], [9, 16, 4, 2], [-3, 4, 1, 16], [0, 16, 0, 16], [1 << 30, -5, 7, 1 << 30]):
        b.start_d.copy_(torch.tensor(start, dtype=torch.int32))
        out = torch.full_like(q, 7.0)
        c.attend(q, max_new=8, out=out)
        with pytest.raises(RuntimeError, match="BAD_LENGTH"):
            c.check()
        assert (out == 7.0).all()
        c.status.zero_()
    b.start_d.copy_(torch.from_numpy(b.start.astype(np.int32)))
    attend_close(b, c.attend(q, max_new=8))
    c.check()


def test_rows_counted_too_often_are_not_walked():
    # every second sequence goes back over all rows: 128 x 2048 x 8 items of 5 units and 609 to 640 tiles (a row
    # sees 38 913 to 40 960 keys), 1.32e9 units, more than the 2^30 - 1 that a line holds
    from sequence_decode_step_gb300 import PagedKV
    n, seqs = 2048, 256
    i32 = {"dtype": torch.int32, "device": "cuda"}
    k = torch.zeros(1, 8, 16, 64, dtype=torch.bfloat16, device="cuda")
    c = PagedKV(k, k.clone(), torch.zeros(seqs, 2560, **i32), torch.full((seqs,), 40960, **i32),
                torch.tensor([0, n] * 128 + [0], **i32))
    out = torch.full((n, 64, 64), 7.0, device="cuda")
    c.attend(torch.zeros(n, 64, 64, device="cuda"), out=out)
    with pytest.raises(RuntimeError, match="BAD_LENGTH"):
        c.check()
    assert (out == 7.0).all()


def test_tensors_that_do_not_fit_are_refused():
    from sequence_decode_step_gb300 import PagedKV
    b = Batch([(1, 20)], 4, 2, 64, 16, "f32", "bf16", seed=53)
    c = b.cache()
    q = b.q.cuda()
    with pytest.raises(ValueError):
        c.attend(q.double())
    with pytest.raises(ValueError):
        c.attend(q.cpu())
    with pytest.raises(ValueError):
        c.attend(q, out=torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        c.append(b.qkv.cuda()[:, ::2], 4)
    with pytest.raises(ValueError):
        c.append(b.qkv.cuda(), 4, positions=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        g = torch.ones(64, dtype=torch.float16, device="cuda")
        c.append(b.qkv.cuda(), 4, q_norm=g, k_norm=g)
    with pytest.raises(ValueError):
        PagedKV(b.kd, b.vd, b.table_d.long(), b.len_d, b.start_d)
    with pytest.raises(ValueError):
        PagedKV(b.kd, b.vd, b.table_d, b.len_d, b.start_d, prefix_pages=b.len_d, prefix_len=17)


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("seqs,nq,prefix,cols", [
    ([(1, 700), (1, 33), (1, 4000)], 4, 0, 1), ([(1, 700), (1, 33)], 16, 2000, 1),
    ([(30, 700), (0, 3), (9, 60)], 16, 0, 2048), ([(150, 0), (1, 900), (6, 9)], 16, 3000, 2048)])
def test_waits_that_give_up(act, kv, seqs, nq, prefix, cols):
    # every wait gives up at once: the call ends and reports it, and its workspace serves the next call,
    # on decode kernels and on tensor-core tiles, with items split over several CTAs
    from sequence_decode_step_gb300 import _binding as B
    b = Batch(seqs, nq, 2, 64, 16, act, kv, prefix=prefix, seed=113, extra_cols=cols)
    new = int(b.new.max())
    c = b.cache(wait_limit_us=B.QW_PAGED_WAIT_NONE)
    c.attend(b.q.cuda(), max_new=new)
    with pytest.raises(RuntimeError, match="TIMEOUT"):
        c.check()
    d = b.cache(workspace=c.workspace)
    attend_close(b, d.attend(b.q.cuda(), max_new=new))
    d.check()


def test_queries_of_another_head_size_are_refused():
    b = Batch([(1, 20), (1, 5)], 4, 2, 128, 16, "f32", "bf16", seed=137)
    c = b.cache()
    q = b.q.cuda()
    for bad in (q.view(2, 8, 64), q.view(2, 2, 256), q.view(2, 1, 512), q.view(-1), q.view(2, 4, 2, 64),
                torch.zeros(2, 4 * 128 + 64, device="cuda")):
        with pytest.raises(ValueError, match="n_q_heads"):
            c.attend(bad)
    attend_close(b, c.attend(q))
    attend_close(b, c.attend(q.view(2, 512)))
    c.check()


@pytest.mark.parametrize("act,kv", TYPES)
@pytest.mark.parametrize("seqs,prefix,cols", [([(1, 4000), (1, 900), (1, 33)], 2000, 1),
                                              ([(60, 3000), (1, 900), (30, 9)], 3000, 2048)])
def test_waits_that_give_up_now_and_then(act, kv, seqs, prefix, cols):
    # a limit of a microsecond, which some waits keep and others do not: every call ends, one that reports
    # nothing is right, and the workspace serves the next call
    b = Batch(seqs, 16, 2, 64, 16, act, kv, prefix=prefix, seed=173, extra_cols=cols)
    ref, q, new = b.attend(), b.q.cuda(), int(b.new.max())
    c = b.cache(wait_limit_us=1)
    d = b.cache(workspace=c.workspace)
    for _ in range(10):
        got = c.attend(q, max_new=new)
        if int(c.status.item()) == 0:
            attend_close(b, got, ref)
        c.status.zero_()
        attend_close(b, d.attend(q, max_new=new), ref)
    d.check()
