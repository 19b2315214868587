"""GPU attention over a paged cache behind a shared prefix against a 64-bit
oracle, elementwise within a bound made of the roundings that the operator is
allowed (see kv_util.AttnCase.bounds)."""
import numpy as np
import pytest
import torch

from gpu_util import note
from kv_util import AttnCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8"), ("fp16", "fp8")])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 144, 256])
def test_types_and_head_widths(dtype, cache, D):
    note(f"attn {dtype} {cache} D={D}")
    AttnCase([40, 1, 129, 300], [1, 1, 2, 1], 8, 2, D, dtype, cache, prefix=75, seed=D).check()


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 1), (12, 12), (33, 1), (28, 4), (64, 2)])
def test_head_layouts(Hq, Hk):
    note(f"attn heads {Hq}/{Hk}")
    AttnCase([37, 200, 65], [1, 3, 1], Hq, Hk, 64, "fp16", prefix=33, seed=Hq).check()


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000])
def test_lengths_of_one_request(n):
    note(f"attn one request of {n}")
    AttnCase([n], [1], 4, 1, 64, "bf16", seed=n).check()


@pytest.mark.parametrize("prefix", [1, 15, 16, 17, 64, 129, 1030])
@pytest.mark.parametrize("joined", [False, True])
def test_prefix_lengths(prefix, joined):
    """Both ways of reading the prefix: as one product for all, and request by request."""
    lens = [3, 1, 20, 2, 9, 1] if not joined else [900, 1100, 1000]
    note(f"attn prefix {prefix} own {lens}")
    AttnCase(lens, [1] * len(lens), 8, 2, 128, "bf16", prefix=prefix, seed=prefix).check()


@pytest.mark.parametrize("block", [1, 3, 8, 24, 64, 200])
@pytest.mark.parametrize("head_major", [False, True])
def test_pages(block, head_major):
    """Pages smaller and larger than a tile of keys, of odd sizes, both layouts, with a gap between pages."""
    note(f"attn block {block} head_major {head_major}")
    AttnCase([150, 77, 201], [1, 2, 1], 8, 2, 64, "fp16", block=block, prefix=90, head_major=head_major, pad=48, seed=block).check()


@pytest.mark.parametrize("lens,new", [([40], [40]), ([300], [300]), ([130, 1, 260], [130, 1, 200]), ([500, 30, 31, 700], [129, 1, 30, 3]),
                                      ([64, 128, 192], [64, 128, 64])])
@pytest.mark.parametrize("prefix", [0, 100])
def test_prompts(lens, new, prefix):
    """Several new tokens of a request see one another in order; tiles of many rows next to single tokens."""
    note(f"attn prompts {lens} {new} prefix {prefix}")
    AttnCase(lens, new, 8, 2, 64, "bf16", prefix=prefix, seed=7).check()


@pytest.mark.parametrize("dtype,cache,D", [("bf16", "bf16", 128), ("fp16", "fp8", 128), ("bf16", "bf16", 256), ("fp16", "fp16", 80)])
def test_prompt_types(dtype, cache, D):
    note(f"attn prompt types {dtype} {cache} {D}")
    AttnCase([333, 90], [333, 77], 4, 2, D, dtype, cache, prefix=40, seed=3).check()


def test_many_rows_share_a_prefix():
    """More rows than a tile behind one prefix, cut into parts, with requests that have no new token."""
    note("attn 50 requests")
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(1, 60, 50)]
    new = [int(rng.integers(0, 2)) for _ in lens]
    AttnCase(lens, new, 16, 2, 128, "bf16", prefix=2100, seed=5).check()


@pytest.mark.parametrize("softcap", [1.0, 30.0])
def test_softcap(softcap):
    note(f"attn softcap {softcap}")
    AttnCase([100, 33, 257], [1, 2, 40], 8, 4, 64, "fp16", prefix=50, softcap=softcap, q_gain=4.0, seed=2).check()


def test_sharp_scores():
    """Scores far apart: one key takes all the weight, and the maximum rises late."""
    c = AttnCase([700], [1], 4, 1, 128, "bf16", seed=11, q_gain=20.0)
    note("attn sharp scores")
    c.check()


def test_rows_without_keys():
    """No prefix, and an own length shorter than the new tokens: the first ones see nothing."""
    note("attn empty rows")
    c = AttnCase([2, 0, 5], [5, 3, 1], 4, 2, 64, "bf16", seed=1)
    got, ls, _ = c.check()
    assert (got[:3] == 0).all() and np.isneginf(ls[:3]).all()
    assert (got[5:8] == 0).all() and np.isneginf(ls[5:8]).all()


def test_rows_without_own_keys_see_the_prefix():
    note("attn prefix only")
    AttnCase([2, 0, 5], [5, 3, 1], 4, 2, 64, "bf16", seed=1, prefix=70).check()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_unseen_values_never_reach_a_row(cache):
    """NaN and infinities in later tokens of a prompt, in the rest of the last
    page, in pages nobody holds: rows that do not see them are as without them,
    rows that do get NaN or the infinity as the formula says."""
    note(f"attn unseen {cache}")
    c = AttnCase([70, 300], [70, 200], 4, 2, 64, "bf16", cache, seed=4, prefix=20)
    clean, _, _ = c.run()
    k, v = c.store
    P = c.block

    def at(r, i):
        return int(c.table[r, i // P]), i % P

    raw = [x.view(torch.uint8) if cache == "fp8" else x.view(torch.int16) for x in c.store]
    nan = 0x7F if cache == "fp8" else 0x7FC0
    for side in raw:  # beyond the lengths
        held = {(int(b), s) for i in range(c.prefix) for b, s in [(c.prefix_ids[i // P], i % P)]}
        held |= {at(r, i) for r in range(2) for i in range(c.kv_lens[r])}
        for b in range(c.nb):
            for s in range(P):
                if (b, s) not in held:
                    side[b, s] = nan
    got, _, _ = c.run()
    assert np.array_equal(got, clean)
    b, s = at(0, 50)     # token 50 of the first prompt (70 new tokens): rows 0..49 do not see it
    raw[1][b, s, 0, 3] = nan
    b, s = at(1, 150)    # token 150 of the second request: its new token 50
    raw[1][b, s, 1, 60] = nan if cache == "fp8" else 0x7F80  # +inf
    raw[0][b, s, 0, :] = nan
    got, _, _ = c.run()
    want = clean.copy()
    want[50:70, 0:2, 3] = np.nan
    want[70 + 50:, 0:2, :] = np.nan
    want[70 + 50:, 2:4, 60] = np.nan if cache == "fp8" else np.inf
    np.testing.assert_array_equal(got, want)


def test_bounds_larger_than_the_lengths():
    """max_new, max_kv and total_kv only size the launch."""
    note("attn loose bounds")
    c = AttnCase([40, 333, 7], [1, 2, 1], 8, 2, 64, "bf16", prefix=50, seed=9)
    c.check(max_new=50, max_kv=5000)
    c.check(max_new=2, max_kv=333, total_kv=380)


def test_padding_rows_are_not_written():
    note("attn padding rows")
    c = AttnCase([40, 333], [1, 2], 8, 2, 64, "bf16", prefix=200, seed=9, total_rows=9, q_pad=16)
    got, ls, args = c.check()
    assert (got[3:] == 7).all() and (ls[3:] == 7).all()
    assert (args[14][:, 8 * 64:] == 7).all()  # the gap between rows


def test_without_lse_and_on_another_stream():
    note("attn other stream")
    c = AttnCase([40, 333], [1, 2], 8, 2, 64, "bf16", prefix=200, seed=9)
    want, _, _ = c.run()
    s = torch.cuda.Stream()
    got, _, _ = c.run(stream=s, lse=False)
    assert np.array_equal(got, want)


def test_pages_outside_the_cache_read_as_zeros():
    """A table entry that is no page: zero keys and values, not a read out of bounds."""
    note("attn bad page ids")
    c = AttnCase([64], [1], 4, 1, 64, "bf16", seed=3)
    zero = AttnCase([64], [1], 4, 1, 64, "bf16", seed=3)
    for side in zero.store:
        side[int(zero.table[0, 1])] = 0
        side[int(zero.table[0, 2])] = 0
    c.table[0, 1], c.table[0, 2] = -5, c.nb
    a, b = c.run()[0], zero.run()[0]
    assert np.array_equal(a, b)


def test_cache_beyond_32_bit_offsets():
    """Pages whose element offsets pass 2^32 (a cache of 9 GiB a side)."""
    note("attn large offsets")
    c = AttnCase([300, 120], [1, 1], 4, 2, 128, "bf16", block=16, seed=6, prefix=60)
    want, wl, args = c.run()
    d, kv, B, T, q, qs, k, v, pre, P, table, width, lens, cu, out, os_, ls, ws, nb, ks, vs = args
    from bit_quantized_gemm_w4a16_amd import hq
    stride = (9 << 30) // 2 // c.nb // 16 * 16
    assert stride * (c.nb - 1) > 1 << 32
    big = []
    for x in (k, v):
        t = torch.empty(stride * c.nb, dtype=torch.bfloat16, device="cuda")
        for i in range(c.nb):
            t[i * stride:i * stride + x[i].numel()] = x[i].reshape(-1)
        big.append(t)
    kv2 = hq.kv_desc(hq.HQ_DT_BF16, c.nb, 16, 2, 128)
    kv2.block_stride = stride
    out.fill_(7)
    hq.hq_attn(d, kv2, B, T, q, qs, big[0], big[1], pre, P, table, width, lens, cu, out, os_, ls, ws, nb)
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy().reshape(want.shape), want)
    assert np.array_equal(ls.double().cpu().numpy(), wl)


@pytest.mark.parametrize("n", [8, 9, 15, 16, 17])
@pytest.mark.parametrize("cache", ["fp16", "fp8"])
def test_drafts(n, cache):
    """Around one and two tiles of 32 rows of a request (4 rows a token), at its own
    keys and at a prefix that few rows share."""
    note(f"attn drafts {n} {cache}")
    AttnCase([n + 200, n, n + 33], [n, n, 1], 8, 2, 64, "fp16", cache, prefix=130, seed=n).check()
    AttnCase([n + 700], [n], 8, 2, 128, "fp16", cache, seed=n).check()
    AttnCase([5, 6], [min(n, 5), 3], 8, 2, 64, "fp16", cache, prefix=700, seed=n).check()


def test_many_requests_of_all_kinds():
    """300 requests with no, one, a few and many new tokens: every token finds its request."""
    note("attn 300 requests")
    rng = np.random.default_rng(3)
    new = [int(x) for x in rng.choice([0, 0, 1, 1, 3, 12, 40], 300)]
    new[0], new[150], new[299] = 0, 150, 33
    lens = [n + int(rng.integers(0, 30)) for n in new]
    AttnCase(lens, new, 4, 1, 16, "bf16", prefix=20, seed=3).check()


def test_very_long_context():
    """More keys than 256 parts of the smallest chunk hold."""
    note("attn 140000 keys")
    AttnCase([140000], [1], 2, 1, 16, "bf16", block=64, seed=8).check()
    AttnCase([3, 1], [1, 1], 1, 1, 16, "fp16", block=64, prefix=150000, seed=8).check()


def test_equal_calls_give_equal_bits():
    note("attn twice")
    c = AttnCase([40, 3000, 700], [1, 2, 90], 8, 2, 128, "bf16", "fp8", prefix=1500, seed=9)
    a, la, _ = c.run()
    for _ in range(3):
        b, lb, _ = c.run()
        assert np.array_equal(a, b) and np.array_equal(la, lb)


def test_graph_replays():
    """A captured call reads lengths and tables as they are at each replay."""
    from bit_quantized_gemm_w4a16_amd import hq
    from kv_util import i32
    note("attn graph")
    c = AttnCase([900, 40, 333], [1, 1, 1], 8, 2, 128, "bf16", prefix=700, seed=12)
    _, _, args = c.run()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            hq.hq_attn(*args)
    for lens in ([900, 40, 333], [512, 1, 2], [0, 0, 77], [900, 40, 333]):
        args[12].copy_(i32(lens))
        args[14].fill_(5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = args[14].clone()
        args[14].fill_(6)
        hq.hq_attn(*args)
        torch.cuda.synchronize()
        assert torch.equal(got, args[14])
        c.kv_lens = lens
        out, lse, parts = c.oracle()
        tol, _ = c.bounds(out, lse, parts)
        assert (np.abs(got[:, :8 * 128].double().cpu().numpy().reshape(out.shape) - out) <= tol).all()


@pytest.mark.parametrize("prefix", [0, 900])
def test_bounds_smaller_than_the_lengths(prefix):
    """A max_new or max_kv that is too small leaves tokens or keys out; the rest is as it should be."""
    note(f"attn tight bounds prefix {prefix}")
    c = AttnCase([40, 700, 90], [1, 50, 20], 8, 2, 64, "bf16", prefix=prefix, seed=9)
    out, lse, parts = c.oracle()
    tol, _ = c.bounds(out, lse, parts)
    got, _, _ = c.run(max_new=30)
    rows = np.r_[0:31, 51:71]  # the first 30 tokens of the second request, all others
    assert (np.abs(got - out) <= tol)[rows].all()
    got, _, _ = c.run(max_kv=64)   # a request's keys from 64 on do not count
    assert (np.abs(got - out) <= tol)[0].all()
    k, v = c.held(0, 1)[:prefix + 64], c.held(1, 1)[:prefix + 64]
    from oracle import kv as okv
    o2, l2, p2 = okv.attention(c.q[1:51].double().numpy(), lambda r: k, lambda r: v, prefix, [64 + 49], [0, 50], float(np.float32(c.scale)))
    t2, _ = c.bounds(o2, l2, p2)
    assert (np.abs(got[1:51] - o2) <= t2).all()


def listed(c, **bounds):
    from bit_quantized_gemm_w4a16_amd import hq
    d, kv = c.descs(**bounds)
    return "listed=1" in hq.hq_attn_plan(d, kv, len(c.new), c.total, c.prefix)[0]


@pytest.mark.parametrize("B,Hq,Hk,D,dtype,cache,prefix,drafts", [
    (7, 8, 2, 64, "bf16", "bf16", 0, 1), (64, 8, 2, 64, "fp16", "fp16", 300, 1), (65, 4, 4, 80, "bf16", "fp8", 0, 9), (200, 8, 1, 64, "bf16", "bf16", 0, 6),
    (20, 16, 2, 128, "bf16", "bf16", 1000, 8), (40, 16, 2, 64, "bf16", "bf16", 100, 20), (130, 4, 1, 256, "fp16", "fp8", 77, 12)])
def test_listed_parts(B, Hq, Hk, D, dtype, cache, prefix, drafts):
    """Lengths that differ, known in sum: the parts are listed on the card.  Requests without new
    tokens, without keys, with one or two tiles of rows, and with more than those hold."""
    note(f"attn listed {B} {Hq}/{Hk} {D} {cache} prefix {prefix}")
    g = np.random.default_rng(B)
    held = g.integers(0, 60, B)
    held[g.integers(0, B, max(B // 16, 1))] = 5000
    held[B // 2], held[-1] = 0, 4999
    new = g.integers(0, drafts + 1, B)
    new[B // 2], new[-1], new[0] = drafts, 1, 0
    c = AttnCase(held.tolist(), new.tolist(), Hq, Hk, D, dtype, cache=cache, prefix=prefix, seed=B)
    total = int(sum(c.kv_lens))
    assert listed(c, total_kv=total) and not listed(c)
    c.check(total_kv=total)
    c.check(total_kv=total + 1000)
