"""hca_shared_attend on the GPU against the definition in 64 bits.

Tolerances, from the arithmetic. Weights are rounded to fp16 (half a step is 2^-11 of a weight; below
2^-14 of the largest one 2^-25 of it, on entries of at most 6 * 2^R with R the largest scale exponent);
operands are exact; the float32 accumulators lose at most 2^-23 of the running sum per 16-entry
step, 2^-13 for 16384 entries, and the logits' errors stay below that again. With
A = sum_j w_j |e_j| of the channel: |error| <= 2^-10 A + 6 n 2^-25 2^R before the output's rounding,
and half a step of bf16, 2^-8 of the value, after it. lse: the logits' error, one part in 2^-23 of
scale * sum |q e| per 16-channel step and a few more, 2^-23 per binade between the rows' scales (a row's
exponent, counted from a common one, is added to its logit), and 2^-20 for the sum of exponentials."""
import math

import numpy as np
import pytest

import oracle
from fp4_kv_cache_csa_b200 import datagen
from gpu_util import dev, host, make_cache

pytestmark = pytest.mark.gpu

E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6]


def random_cache(P, cap, D, fmt=0, n=None, seed=1, block=4, lo=None, hi=None):
    if fmt:
        fp4, sc = datagen.random_cache_bytes_e4m3x16(P * cap, D, seed, 44, scale_lo=lo or 0x1C, scale_hi=hi or 0x2C)
    else:
        fp4, sc = datagen.random_cache_bytes(P * cap, D, seed, 40, scale_lo=lo or 123, scale_hi=hi or 126)
    return make_cache(fp4.reshape(P, cap, D // 2), sc.reshape(P, cap, -1), [cap] * P if n is None else n, block,
                      scale_fmt=fmt)


def entries(c, b, n):
    import torch

    codes, raw = c.fp4[b, :n], c.scale[b, :n]
    lut = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    e = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).reshape(n, raw.shape[1], -1)
    s = raw.view(torch.float8_e4m3fn).double() if c.scale_fmt else torch.exp2(raw.double() - 127)
    return (e * s[..., None]).reshape(n, c.dim)


def reference(c, q, offs, pos, scale, jo=None, jl=None):
    """(out, lse, bound of out before rounding, bound of lse), float64."""
    import torch

    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    A, lse = torch.zeros_like(out), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    dl = torch.full_like(lse, 2.0 ** -20)
    flush = torch.zeros(q.shape[0], dtype=torch.float64, device="cuda")
    filled = c.n_blocks.tolist()
    for b in range(c.batch):
        for i in range(offs[b], offs[b + 1]):
            n = max(min(filled[b], c.capacity), 0)
            if pos is not None:
                n = min(n, max((int(pos[i]) + 1) // c.block, 0))
            if n == 0:
                continue
            e = entries(c, b, n)
            u = scale * (q[i].double() @ e.T)
            lse[i] = torch.logsumexp(u, -1)
            w = torch.exp(u - lse[i][:, None])
            out[i], A[i] = w @ e, w @ e.abs()
            # |scale|: the error of scale * <q, e> has the size of its terms, also where scale is negative
            dl[i] += 2.0 ** -23 * (c.dim / 16 + 8) * abs(scale) * (q[i].double().abs() @ e.abs().T).amax(-1)
            top = e.abs().amax(1)
            top = top[top > 0]
            if len(top):
                dl[i] += 2.0 ** -23 * min(40.0, float(torch.log2(top.max() / top.min())))
            flush[i] = 6 * n * 2.0 ** -25 * float(e.abs().max())
    if jl is not None:
        other = jl.double()
        both = torch.logaddexp(lse, other)
        wa, wb = torch.exp(lse - both).nan_to_num(0), torch.exp(other - both).nan_to_num(0)
        out = wa[..., None] * out + torch.where(wb[..., None] > 0, wb[..., None] * jo.double(), 0)
        A = wa[..., None] * A + torch.where(wb[..., None] > 0, wb[..., None] * jo.double().abs(), 0)
        dl = dl + 2.0 ** -22 * both.abs().nan_to_num(0, 0, 0)
        lse = both
    else:
        dl = dl + 2.0 ** -23 * lse.abs().nan_to_num(0, 0, 0)
    # errors of the two lse shift the shares of the joined parts by at most as much
    return out, lse, 2.0 ** -10 * A + flush[:, None, None] + 2 * dl[..., None] * A, dl


def check(got, lse, c, q, offs, pos, scale, jo=None, jl=None):
    import torch

    out, ref_lse, tol, dl = reference(c, q, offs, pos, scale, jo, jl)
    rows = slice(offs[0], offs[-1])
    err = (got.double() - out).abs()[rows]
    bound = (tol + 2.0 ** -8 * (out.abs() + tol))[rows]
    assert torch.isfinite(got[rows].float()).all()
    bad = err > bound
    assert not bad.any(), (int(bad.sum()), bad.numel(), float(err.max()), float((err / bound.clamp(min=1e-30)).max()))
    if lse is not None:
        fin = torch.isfinite(ref_lse[rows])
        assert torch.equal(torch.isfinite(lse[rows]), fin)
        assert (lse[rows][~fin] == -math.inf).all()
        d = (lse.double() - ref_lse).abs()[rows][fin]
        assert (d <= dl[rows][fin]).all(), float((d / dl[rows][fin]).max())


def run(c, offs, H, pos=None, join=False, seed=3, scale=None, lse=True):
    import torch

    import fp4_kv_cache_csa_b200 as csa

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    Nq = max(offs[-1], 1)
    q = torch.randn(Nq, H, c.dim, generator=g, device="cuda").to(torch.bfloat16)
    jo = jl = None
    if join:
        jo = torch.randn(Nq, H, c.dim, generator=g, device="cuda")
        jl = 5 * torch.randn(Nq, H, generator=g, device="cuda") + 3
        jl[::3, 0] = -math.inf                       # nothing in the other part: its values do not count
        jo[::3, 0] = math.nan
    scale = c.dim ** -0.5 if scale is None else scale
    L = torch.full((Nq, H), 7.0, device="cuda") if lse else None
    got = csa.hca_shared_attend(c, q, dev(np.asarray(offs, np.int32)), None if pos is None else dev(np.asarray(pos, np.int32)),
                                join_out=jo, join_lse=jl, softmax_scale=scale, lse=L)
    assert csa.csa_read_device_status(c) == 0
    check(got, L, c, q, offs, pos, scale, jo, jl)
    return got, L


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("D,H", [(128, 16), (128, 64), (512, 64), (512, 16)])
@pytest.mark.parametrize("n", [1, 127, 128, 129, 1000])
def test_one_slot(D, H, n, fmt):
    run(random_cache(1, n, D, fmt), [0, 5], H, join=n % 2 == 1)


@pytest.mark.parametrize("H", [1, 3, 7, 16, 21, 22, 32, 33, 40, 64])
@pytest.mark.parametrize("D", [128, 512])
def test_head_counts(D, H):
    run(random_cache(2, 300, D, n=[300, 171]), [0, 9, 13], H, join=True)


@pytest.mark.parametrize("D,fmt", [(128, 0), (512, 1)])
def test_slots_of_all_kinds(D, fmt):
    # an empty slot, one without queries, one without both, a count beyond the capacity and one below zero
    c = random_cache(7, 260, D, fmt, n=[260, 0, 5, 0, 999, -4, 131])
    run(c, [0, 3, 5, 5, 5, 70, 71, 75], 16, join=False)
    run(c, [0, 3, 5, 5, 5, 70, 71, 75], 16, join=True)


def test_rows_without_a_slot_are_left_alone():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c = random_cache(2, 140, 128)
    q = dev(datagen.normal_bf16((9, 16, 128), 4, 1))
    out = torch.full((9, 16, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 16), 5.0, device="cuda")
    csa.hca_shared_attend(c, q, dev(np.array([2, 4, 7], np.int32)), out=out, lse=lse)
    check(out, lse, c, q, [2, 4, 7], None, 128 ** -0.5)
    for rows in (slice(0, 2), slice(7, 9)):
        assert (out[rows] == 3).all() and (lse[rows] == 5).all()


@pytest.mark.parametrize("D,H,m", [(128, 16, 4), (512, 64, 4), (512, 24, 128), (128, 64, 1)])
def test_causal(D, H, m):
    n = 517
    c = random_cache(2, n, D, n=[n, 300], block=m)
    # ascending and shuffled positions, before the first block, at block borders, beyond the last block
    rng = np.random.default_rng(5)
    pos = np.concatenate([np.arange(-3, 2 * m), rng.integers(0, n * m, 37), [n * m - 2, n * m - 1, n * m + 5 * m]])
    run(c, [0, len(pos) - 6, len(pos)], H, pos=pos, join=False)
    run(c, [0, len(pos) - 6, len(pos)], H, pos=pos, join=True)


@pytest.mark.parametrize("D,H,P,Nq,n", [(512, 64, 1, 32, 4101), (512, 64, 3, 400, 260), (128, 16, 1, 4, 1024),
                                        (128, 16, 2, 2000, 513), (512, 8, 1, 600, 1537), (512, 64, 1, 1, 16385)])
def test_splits(D, H, P, Nq, n):
    # few groups spread over many CTAs, many groups per CTA, groups cut at every kind of place
    w = np.sort(np.random.default_rng(Nq).integers(0, Nq + 1, P - 1))
    run(random_cache(P, n, D, n=[n - 13 * p for p in range(P)]), [0, *w.tolist(), Nq], H, join=Nq % 2 == 0)


@pytest.mark.parametrize("D,H,Nq,n,causal", [(128, 64, 1301, 300, False), (512, 33, 700, 517, True)])
def test_more_groups_than_the_small_plan_takes(D, H, Nq, n, causal):
    c = random_cache(3, n, D, n=[n, 0, n - 130])
    pos = np.random.default_rng(1).integers(-2, 4 * n + 8, Nq) if causal else None
    run(c, [0, Nq // 2, Nq // 2 + 7, Nq], H, pos=pos, join=causal)


def test_more_slots_than_the_small_plan_takes():
    rng = np.random.default_rng(2)
    P = 1100
    n = rng.integers(0, 140, P)
    queries = rng.integers(0, 3, P)
    queries[[0, -1]] = 0
    run(random_cache(P, 139, 128, n=n.tolist()), [0, *np.cumsum(queries).tolist()], 16, join=True)


def test_against_the_oracle_and_hca_decode_attend():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    D, H, n = 512, 64, 700
    fp4, sc = datagen.random_cache_bytes(n, D, 9, 40, scale_lo=120, scale_hi=127)
    fp4, sc = fp4.reshape(1, n, D // 2), sc.reshape(1, n, D // 32)
    q = datagen.normal_bf16((6, H, D), 9, 1)
    offs, pos = np.array([0, 6], np.int32), np.array([10, 511, 512, 2000, 2799, 9999], np.int32)
    ref, ref_lse = oracle.hca_attend(fp4, sc, [n], offs, pos, q, None, None, None, D ** -0.5, m=4)
    c = make_cache(fp4, sc, [n], 4)
    lse = torch.empty(6, H, device="cuda")
    got = csa.hca_shared_attend(c, dev(q), dev(offs), dev(pos), lse=lse)
    check(got, lse, c, dev(q), [0, 6], pos, D ** -0.5)
    # the decode kernel holds 2e-3 of the row's largest value, this one half a bf16 step on top
    top = np.abs(ref).max(-1, keepdims=True)
    assert np.all(np.abs(got.float().cpu().numpy() - ref) <= 2e-3 * top + 2.0 ** -8 * np.abs(ref) + 1e-30)
    assert np.all(np.abs(host(lse) - ref_lse) <= 1e-3 + 1e-4 * np.abs(ref_lse))
    old = csa.hca_decode_attend(c, dev(q), dev(offs), dev(pos))
    assert np.all(np.abs(got.float().cpu().numpy() - host(old)) <= 4e-3 * top + 2.0 ** -8 * np.abs(ref) + 1e-30)


@pytest.mark.parametrize("fmt,lo,hi", [(0, 90, 140), (0, 1, 60), (1, 0x01, 0x7E)])
def test_scales_of_many_binades(fmt, lo, hi):
    # a row's small groups vanish beside its largest one only below 2^-24 of it, tiny rows beside the others
    run(random_cache(1, 400, 512, fmt, lo=lo, hi=hi), [0, 3], 64, scale=1e-4 if fmt == 0 and hi > 100 else 1e-3)


def test_references_rise():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    # logits that climb by tens of bits from tile to tile, for some columns only, and fall for others
    c = random_cache(1, 1280, 128, seed=6)
    ramp = torch.repeat_interleave(torch.arange(10, device="cuda", dtype=torch.uint8), 128)
    c.scale[0] = (118 + ramp)[:, None]
    run(c, [0, 8], 8, scale=0.5)
    run(c, [0, 8], 8, scale=-2.0)


def test_zero_rows_and_zero_queries():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c = random_cache(1, 300, 512)
    c.fp4.zero_()
    c.scale.zero_()                                   # pooled zero tokens: scale byte 0
    out, lse = run(c, [0, 2], 64)
    assert (out == 0).all() and float((lse - math.log(300)).abs().max()) <= 2e-6 * 6
    c = random_cache(1, 300, 512)
    c.scale[0, 100:200] = 0
    c.fp4[0, 100:200] = 0
    q = torch.zeros(2, 64, 512, dtype=torch.bfloat16, device="cuda")
    got = csa.hca_shared_attend(c, q, dev(np.array([0, 2], np.int32)))
    check(got, None, c, q, [0, 2], None, 512 ** -0.5)


def test_extreme_queries_stay_in_their_columns():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c = random_cache(1, 500, 128)
    q = dev(datagen.normal_bf16((4, 16, 128), 4, 1))
    want = csa.hca_shared_attend(c, q, dev(np.array([0, 4], np.int32)))
    bad = q.clone()
    bad[1, 3] = math.nan
    bad[2, 5, 7] = math.inf
    bad[0, 0] = 1e-38                                 # its logits vanish: the mean of the entries
    bad[0, 1] = bad[0, 1] * 1e30
    got = csa.hca_shared_attend(c, bad, dev(np.array([0, 4], np.int32)))
    assert torch.isnan(got[1, 3]).all() and not torch.isfinite(got[2, 5]).any()
    touched = torch.zeros(4, 16, dtype=torch.bool, device="cuda")
    for i, h in ((1, 3), (2, 5), (0, 0), (0, 1)):
        touched[i, h] = True
    assert torch.equal(got[~touched], want[~touched])
    e = entries(c, 0, 500)
    mean, A = e.mean(0), e.abs().mean(0)
    assert ((got[0, 0].double() - mean).abs() <= 2.0 ** -10 * A + 6 * 500 * 2.0 ** -25 + 2.0 ** -8 * mean.abs()).all()
    assert torch.isfinite(got[0, 1].float()).all()    # one entry takes all the weight


def test_nan_behind_the_visible_blocks():
    import torch

    # blocks behind n_blocks are never read, whatever their bytes
    c = random_cache(2, 256, 128, fmt=1, n=[200, 129])
    c.scale[0, 200:] = 0x7F
    c.scale[1, 129:] = 0x7F
    c.fp4[0, 200:] = 0x77
    run(c, [0, 5, 9], 16)


@pytest.mark.parametrize("H", [16, 64])
def test_a_nan_of_the_other_part_stays_one(H):
    import torch

    import fp4_kv_cache_csa_b200 as csa

    # slot 0 has no blocks, slot 1 some, slot 2 so many that several thread blocks share the group
    c = random_cache(3, 20000, 512, n=[0, 300, 20000])
    q = dev(datagen.normal_bf16((6, H, 512), 4, 1))
    offs = dev(np.array([0, 2, 4, 6], np.int32))
    jo, jl = torch.ones(6, H, 512, device="cuda"), torch.zeros(6, H, device="cuda")
    jl[::2, 3] = math.nan
    lse = torch.empty(6, H, device="cuda")
    out = csa.hca_shared_attend(c, q, offs, join_out=jo, join_lse=jl, lse=lse)
    assert torch.equal(lse.isnan(), jl.isnan())
    assert torch.equal(out.isnan(), jl.isnan()[..., None].expand(out.shape))


def test_offsets_beyond_32_bits():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    cap, P = 1 << 19, 33                              # slot 32 lies behind 2^32 bytes of codes
    c = csa.Cache.allocate(P, cap, 512, 4)
    part = random_cache(1, 1000, 512)
    c.fp4[P - 1, :1000], c.scale[P - 1, :1000] = part.fp4[0], part.scale[0]
    c.n_blocks[P - 1] = 1000
    q = dev(datagen.normal_bf16((2, 64, 512), 4, 1))
    offs = dev(np.array([0] * P + [2], np.int32))
    assert torch.equal(csa.hca_shared_attend(c, q, offs),
                       csa.hca_shared_attend(part, q, dev(np.array([0, 2], np.int32))))
    assert csa.csa_read_device_status(c) == 0


def test_same_inputs_same_bits_graph_and_stream():
    import torch

    import fp4_kv_cache_csa_b200 as csa

    c, H = random_cache(2, 900, 512), 64
    offs = dev(np.array([0, 6, 11], np.int32))
    q = dev(datagen.normal_bf16((11, H, 512), 4, 1))
    want = csa.hca_shared_attend(c, q, offs)
    assert torch.equal(csa.hca_shared_attend(c, q, offs), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = csa.hca_shared_attend(c, q, offs, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(csa.hca_shared_attend_workspace(c, 11, H), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.empty_like(q), torch.empty_like(q)], []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            csa.hca_shared_attend(c, q, offs, out=o, workspace=ws)
        graphs.append(g)
    for seed in (2, 3):
        q.copy_(dev(datagen.normal_bf16((11, H, 512), 4, seed)))
        c.n_blocks.fill_(900 - 130 * seed)            # the replay reads the counts of its own time
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = csa.hca_shared_attend(c, q, offs)
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("heads", [16, 64])
def test_continuations_of_one_prompt(heads):
    """The operators together: queries and newest tokens rotated, the prompt's slot shared by all
    continuations, their own blocks in slots forked from a template, outputs turned back; against one
    softmax over everything in float64."""
    import torch

    import fp4_kv_cache_csa_b200 as csa

    D, R, S, n, own = 512, 64, 5, 777, 40
    prompt = random_cache(1, n, D, seed=8, block=4)
    tails = random_cache(S + 1, own + 3, D, seed=9, n=[own] + [0] * S, block=4)
    inv = csa.csa_rotary_frequencies(R, scaling=csa.CSA_ROPE_SCALE_PARTS, factor=4.0, original_len=1024)[0].cuda()
    i32 = lambda v: dev(np.asarray(v, np.int32))  # noqa: E731
    pos = i32([4 * (n + own) + s for s in range(S)])
    # every continuation starts from the same own blocks
    csa.csa_cache_copy(tails, tails, i32([0] * S), i32(range(1, S + 1)))
    q = csa.csa_rotary(dev(datagen.normal_bf16((S, heads, D), 1, 2)), pos, inv)
    win = csa.csa_rotary(dev(datagen.normal_bf16((S * 8, D), 1, 3)), torch.repeat_interleave(pos, 8), inv)
    qo = i32([0, 0, 1, 2, 3, 4, 5])
    part_lse = torch.empty(S, heads, device="cuda")
    part = csa.hca_decode_attend(tails, q, qo, i32([4 * own - 1] * S), win, dev(np.arange(0, 8 * S, 8, dtype=np.int64)),
                                 i32([8] * S), lse=part_lse)
    lse = torch.empty(S, heads, device="cuda")
    out = csa.hca_shared_attend(prompt, q, i32([0, S]), join_out=part, join_lse=part_lse, lse=lse)
    back = csa.csa_rotary(out, pos, inv, inverse=True)
    assert csa.csa_read_device_status(tails) == 0 and csa.csa_read_device_status(prompt) == 0
    for s in range(S):
        e = torch.cat((entries(prompt, 0, n), entries(tails, 0, own), win[8 * s:8 * s + 8].double()))
        u = D ** -0.5 * (q[s].double() @ e.T)
        total = torch.logsumexp(u, -1)
        w = torch.exp(u - total[:, None])
        want = w @ e
        top = want.abs().amax(-1, keepdim=True)
        # the decode call's 2e-3 of the row's largest value, and half a step of bf16
        assert ((out[s].double() - want).abs() <= 2e-3 * top + 2.0 ** -8 * want.abs()).all()
        assert ((lse[s].double() - total).abs() <= 1e-3 + 1e-4 * total.abs()).all()
        ang = float(pos[s]) * inv.double()
        z = torch.complex(out[s, :, D - R::2].double(), out[s, :, D - R + 1::2].double()) * torch.polar(torch.ones_like(ang), -ang)
        turned = torch.stack((z.real, z.imag), -1).flatten(-2)
        # 9 steps of 2^-24 on |a| + |b| for the rotation, half a bf16 step for its output
        assert ((back[s, :, D - R:].double() - turned).abs()
                <= 2.0 ** -8 * turned.abs() + 9 * 2.0 ** -24 * 4 * float(top.max())).all()
        assert torch.equal(back[s, :, :D - R], out[s, :, :D - R])
