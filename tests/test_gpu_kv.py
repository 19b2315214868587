"""GPU slot maps, rotary table, and rotation with the cache write against the
64-bit definitions."""
import numpy as np
import pytest
import torch

import oracle
from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from kv_util import DT, HQ_DT, TINY, U, i32
from oracle import kv as okv

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# slot maps
# ---------------------------------------------------------------------------

def run_slots(cached, new, P, free, table, T_cap, first=0):
    B = len(cached)
    t = i32(table) if B else None
    dev = dict(cu=torch.full((B + 1,), 77, dtype=torch.int32).cuda(), kv=torch.full((max(B, 1),), 77, dtype=torch.int32).cuda(),
               pos=torch.full((max(T_cap, 1),), 77, dtype=torch.int32).cuda(), slots=torch.full((max(T_cap, 1),), 77, dtype=torch.int64).cuda(),
               taken=torch.full((1,), 77, dtype=torch.int32).cuda())
    hq.hq_kv_slots(P, B, T_cap, i32(cached) if B else None, i32(new) if B else None, i32(free) if len(free) else None, len(free), t,
                   np.shape(table)[1] if B else 0, dev["cu"], dev["kv"], dev["pos"], dev["slots"], dev["taken"], first_pos=first)
    torch.cuda.synchronize()
    n = lambda x: x.cpu().numpy()  # noqa: E731
    return n(dev["cu"]), n(dev["kv"])[:B], n(t) if B else table, n(dev["pos"])[:T_cap], n(dev["slots"])[:T_cap], int(dev["taken"][0])


def check_slots(cached, new, P, free, table, T_cap, first=0):
    got = run_slots(cached, new, P, free, table, T_cap, first)
    want = okv.slots(cached, new, free, table, P, T_cap, first)
    for g, w, name in zip(got, want, ("cu_new", "kv_lens", "block_table", "positions", "slots", "taken")):
        np.testing.assert_array_equal(np.asarray(g, dtype=np.int64), np.asarray(w, dtype=np.int64), err_msg=name)


@pytest.mark.parametrize("B", [1, 2, 63, 255, 256, 257, 1000, 4096])
@pytest.mark.parametrize("P", [1, 16, 24])
def test_slots(B, P):
    note(f"slots B={B} P={P}")
    rng = np.random.default_rng([B, P])
    cached = rng.integers(0, 200 if B < 1000 else 40, B)
    new = rng.integers(0, 40 if B < 1000 else 4, B)
    cached[rng.random(B) < 0.2] = 0
    width = int(max(-(-(cached + new) // P))) + 1
    table = rng.integers(0, 1 << 20, (B, width))
    need = int((-(-(cached + new) // P) + (-cached // P)).sum())
    check_slots(cached, new, P, rng.permutation(need + 5) + 3, table, int(new.sum()) + 7, first=11)


def test_slots_long_prompt_and_large_ids():
    """A prompt over many pages, and page ids whose slots pass 2^31."""
    note("slots long prompt")
    table = np.full((3, 2000), 40000000)
    check_slots([5000, 0, 17], [1, 20000, 0], 64, np.arange(1000) + 50000000, table, 20001)


def test_slots_without_free_pages_or_table_room():
    note("slots short of pages")
    check_slots([10, 3, 0], [30, 30, 30], 8, [5, 6, 7], np.full((3, 3), 9), 100)
    check_slots([10, 3, 0], [30, 30, 30], 8, [], np.full((3, 3), 9), 10)


def test_slots_empty_and_negative():
    note("slots empty")
    check_slots([], [], 16, [1], np.zeros((0, 0)), 4)
    check_slots([0, 0], [0, 0], 16, [1, 2], np.zeros((2, 2)), 0)
    check_slots([-3, 5, -1], [4, -2, 2], 4, [8, 9, 10], np.zeros((3, 4)), 9)


def test_slots_saturate():
    """Sums beyond 2^31-1 saturate; nothing is written out of bounds."""
    note("slots saturate")
    big = 2 ** 31 - 1
    cu, kv, _, pos, slots, _ = run_slots([big, 5], [big, big], 16, [1, 2], np.full((2, 2), 3), 40)
    assert cu.tolist() == [0, big, big] and kv.tolist() == [big, big]
    assert (slots == -1).all() and (pos == big).all()


# ---------------------------------------------------------------------------
# rotary table
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("scaling,kind", [("none", 0), ("linear", 1), ("ntk", 2), ("parts", 3)])
@pytest.mark.parametrize("rot,first,count", [(16, 0, 1), (64, 0, 3001), (128, 130000, 77), (256, 2 ** 31 - 9, 9), (96, 1000003, 50)])
def test_rope_table(scaling, kind, rot, first, count):
    """Two fp32 roundings (the angle in turns, half of 2^-24, and the value) and the
    library's cos and sin (2 units): below 2^-21 of the gain, at every position
    whose 64-bit turns are good to 2^-26 (2^53 / 2^26 = 2^27); beyond that the
    oracle's own angle, reduced from radians, is the limit."""
    note(f"rope table {scaling} rot={rot} first={first}")
    p = dict(base=500000.0, factor=4.0 if kind else 1.0, context=4096.0)
    desc = hq.rope_desc(rot, p["base"], scaling=kind, factor=p["factor"], context=p["context"])
    t = torch.full((count, rot), 9.0).cuda()
    hq.hq_rope_table(desc, first, count, t)
    torch.cuda.synchronize()
    want = okv.rope_table(rot, first, count, scaling=scaling, **p)
    err = np.abs(t.double().cpu().numpy() - want).max()
    assert err <= 1.2 * 2.0 ** -21 + (first + count) * 2.0 ** -51, err


def test_rope_table_given_attention_factor():
    note("rope table factor")
    desc = hq.rope_desc(64, scaling=hq.HQ_ROPE_PARTS, factor=8.0, context=2048, slow=2.0, fast=20.0, attn_factor=1.5)
    t = torch.zeros(100, 64).cuda()
    hq.hq_rope_table(desc, 0, 100, t)
    torch.cuda.synchronize()
    want = okv.rope_table(64, 0, 100, scaling="parts", factor=8.0, context=2048, slow=2.0, fast=20.0, attn_factor=1.5)
    assert np.abs(t.double().cpu().numpy() - want).max() <= 1.5 * 2.0 ** -21


# ---------------------------------------------------------------------------
# rotation and cache write
# ---------------------------------------------------------------------------

def rope_case(T, Hq, Hk, D, rot, dtype, cache, interleaved, block=16, head_major=False, seed=0, in_place=False, special=False):
    g = torch.Generator().manual_seed(seed)
    row = (Hq + 2 * Hk) * D
    qkv = torch.randn(T, row + 8, generator=g).to(DT[dtype])
    if special:
        qkv[0, Hq * D] = float("inf")
        qkv[0, Hq * D + Hk * D] = float("nan")
        qkv[0, Hq * D + Hk * D + 1] = float("-inf")
    ang = torch.rand(50, rot // 2, generator=g) * 6.28
    table = torch.cat([ang.cos(), ang.sin()], 1)
    pos = torch.randint(-3, 56, (T,), generator=g)
    nb = T // block + 3
    slots = torch.randperm(nb * block, generator=g)[:T]
    if T > 3:
        slots[1], slots[2] = -1, nb * block  # not written
    scales = [(4 + torch.rand(Hk, generator=g)) / 448 for _ in range(2)] if cache == "fp8" else [None, None]
    shape = (nb, Hk, block, D) if head_major else (nb, block, Hk, D)
    store = [torch.zeros(shape).to(DT[cache]) + torch.zeros(()).to(DT[cache]) if cache != "fp8" else torch.zeros(shape).to(DT[cache]) for _ in range(2)]
    x = qkv.cuda()
    q_out = x if in_place else torch.zeros(T, Hq * D, dtype=DT[dtype]).cuda()
    kc, vc = (s.cuda() for s in store)
    kv = hq.kv_desc(HQ_DT[cache], nb, block, Hk, D, head_major=head_major)
    stride = x.shape[1]
    sc = [None if s is None else s.cuda() for s in scales]
    hq.hq_rope_kv(hq.rope_desc(rot, interleaved=interleaved), kv, HQ_DT[dtype], T, Hq, x, stride, x[:, Hq * D:], stride,
                  x[:, (Hq + Hk) * D:], stride, i32(pos), table.cuda(), 50, slots.cuda(), q_out, stride if in_place else Hq * D, kc, vc, *sc)
    torch.cuda.synchronize()
    h = qkv[:, :row].double().numpy().reshape(T, Hq + 2 * Hk, D)
    rows = table.double().numpy()[np.clip(pos.numpy(), 0, 49)]
    with np.errstate(invalid="ignore"):
        turned = okv.rope(h[:, :Hq + Hk], rows, rot, interleaved)
    want_q = turned[:, :Hq]
    got_q = q_out[:, :Hq * D].double().cpu().numpy().reshape(T, Hq, D)
    # a pair's two fp32 products and their difference, then one rounding
    part = np.abs(okv.rope(np.abs(h[:, :Hq]), np.abs(rows) * np.concatenate([np.ones(rot // 2), -np.ones(rot // 2)]), rot, interleaved))
    tol = U[dtype] * np.abs(want_q) * 1.01 + 2.0 ** -22 * (part + np.abs(h[:, :Hq]).max()) + TINY[dtype]
    assert (np.abs(got_q - want_q) <= tol).all()
    for side, (got, want) in enumerate(((kc, turned[:, Hq:]), (vc, h[:, Hq + Hk:]))):
        got = got.cpu()
        got = got.permute(0, 2, 1, 3) if head_major else got
        got = got.double().numpy().reshape(nb * block, Hk, D)
        expect, touched = np.zeros_like(got), np.zeros(nb * block, dtype=bool)
        for t in range(T):
            s = int(slots[t])
            if 0 <= s < nb * block:
                expect[s], touched[s] = want[t], True
        assert (got[~touched] == 0).all()
        e, y = expect[touched], got[touched]
        if cache == "fp8":
            e = np.clip(e / scales[side].double().numpy()[:, None], -448, 448)
        u = U[cache]
        nan = np.isnan(e)
        assert np.isnan(y[nan]).all() and not np.isnan(y[~nan]).any()
        fin = np.isfinite(e)
        assert (y[np.isinf(e)] == e[np.isinf(e)]).all()
        top = np.abs(e[fin]).max() if fin.any() else 0
        assert (np.abs(y[fin] - e[fin]) <= u * np.abs(e[fin]) * 1.01 + 2.0 ** -21 * top + TINY[cache]).all()


@pytest.mark.parametrize("T", [1, 5, 33, 700])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8"), ("fp16", "fp8")])
def test_rope_kv_types(T, interleaved, dtype, cache):
    note(f"rope kv T={T} {dtype} {cache} interleaved={interleaved}")
    rope_case(T, 8, 2, 64, 64, dtype, cache, interleaved, seed=T)


@pytest.mark.parametrize("Hq,Hk,D,rot", [(1, 1, 16, 16), (5, 1, 80, 32), (32, 32, 80, 80), (3, 3, 256, 64), (64, 8, 128, 128), (7, 7, 96, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_kv_shapes(Hq, Hk, D, rot, interleaved):
    note(f"rope kv {Hq}/{Hk} D={D} rot={rot}")
    rope_case(37, Hq, Hk, D, rot, "bf16", "bf16", interleaved, block=24, head_major=True, seed=D)


@pytest.mark.parametrize("block", [1, 7, 64])
def test_rope_kv_pages_in_place(block):
    note(f"rope kv in place block={block}")
    rope_case(100, 8, 2, 64, 32, "fp16", "fp16", False, block=block, in_place=True)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_rope_kv_special_values(cache):
    """Infinities saturate in E4M3 and stay in 16 bits, NaN stays NaN (rotated pairs of an infinity too)."""
    note(f"rope kv special {cache}")
    rope_case(6, 2, 1, 32, 16, "bf16", cache, False, special=True)


def test_rope_kv_codes_match_the_oracle_encoder():
    """Values that pass through unrotated: the E4M3 codes are the oracle's codes of x / scale, bit for bit."""
    note("rope kv codes")
    T, Hk, D = 64, 2, 32
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(T, 3 * Hk * D, generator=g) * torch.logspace(-3, 3, T)[:, None]).to(torch.bfloat16)
    sc = torch.tensor([0.013, 0.37])
    kc, vc = (torch.zeros(4, 16, Hk, D, dtype=torch.uint8).cuda() for _ in range(2))
    d = x.cuda()
    table = torch.cat([torch.ones(1, 8), torch.zeros(1, 8)], 1).cuda()
    hq.hq_rope_kv(hq.rope_desc(16), hq.kv_desc(hq.HQ_DT_FP8_E4M3, 4, 16, Hk, D), hq.HQ_DT_BF16, T, Hk, d, 3 * Hk * D, d[:, Hk * D:], 3 * Hk * D,
                  d[:, 2 * Hk * D:], 3 * Hk * D, i32(np.zeros(T)), table, 1, torch.arange(T).cuda(), torch.zeros(T, Hk * D, dtype=torch.bfloat16).cuda(),
                  Hk * D, kc, vc, sc.cuda(), sc.cuda())
    torch.cuda.synchronize()
    for got, lo in ((kc, Hk * D), (vc, 2 * Hk * D)):
        v = x[:, lo:lo + Hk * D].float().reshape(T, Hk, D) / sc[:, None]
        v = v.clamp(-448, 448).numpy()
        want = np.array([oracle.e4m3_encode(float(a)) for a in v.reshape(-1)], dtype=np.uint8).reshape(T, Hk, D)
        np.testing.assert_array_equal(got.cpu().numpy().reshape(T, Hk, D), want)
