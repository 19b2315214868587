"""GPU attention on each way that a call can be cut (prefix as one product or walked
by each request; keys in one part or several; few and many rows), each test
with the plan that it is for, against 64 bits on the same inputs."""
import re

import numpy as np
import pytest
import torch

from bit_quantized_gemm_w4a16_amd import hq
from gpu_util import note
from kv_util import AttnCase

pytestmark = pytest.mark.gpu


class Case(AttnCase):
    """The oracle in torch's 64 bits on the card, a request and a key head at a time."""

    def oracle(self):
        T, G = self.total, self.Hq // self.Hk
        f64 = lambda x: torch.as_tensor(x, dtype=torch.float64).cuda()  # noqa: E731
        scale, cap = float(np.float32(self.scale)), float(np.float32(self.softcap))
        out, mass = f64(np.zeros((T, self.Hq, self.D))), f64(np.zeros((T, self.Hq, self.D)))
        lse = f64(np.full((T, self.Hq), -np.inf))
        qk, seen, vmax = (f64(np.zeros((T, self.Hq))) for _ in range(3))
        for r, n in enumerate(self.new):
            if not n or not self.prefix + self.kv_lens[r]:
                continue
            t0 = int(self.cu[r])
            k, v = f64(self.held(0, r)), f64(self.held(1, r))
            sees = self.prefix + (self.kv_lens[r] - n + 1 + torch.arange(n, device="cuda")).clamp(min=0)
            seen[t0:t0 + n] = sees[:, None].double()
            hide = (torch.arange(len(k), device="cuda")[None] >= sees[:, None]).repeat_interleave(G, 0)
            some = (sees > 0).repeat_interleave(G)[:, None]
            for h in range(self.Hk):
                q = f64(self.q[t0:t0 + n, h * G:(h + 1) * G]).reshape(n * G, self.D)
                kt, vh = k[:, h].t().contiguous(), v[:, h].contiguous()
                s = torch.mm(q, kt) * scale
                if cap:
                    s = cap * torch.tanh(s / cap)
                s = s.masked_fill(hide, -torch.inf)
                m = s.amax(1, keepdim=True)
                p = torch.exp(s - m.where(some, 0.0))
                total = p.sum(1, keepdim=True)
                p = (p / total).where(some, 0.0)
                top = torch.cat([vh.new_zeros(1), vh.abs().amax(1).cummax(0).values])  # of the first keys
                for to, x in ((out, torch.mm(p, vh)), (mass, torch.mm(p, vh.abs())), (lse, m + torch.log(total)),
                              (qk, (torch.mm(q.abs(), kt.abs()) * scale).masked_fill(hide, 0.0).amax(1)), (vmax, top[sees.repeat_interleave(G)])):
                    to[t0:t0 + n, h * G:(h + 1) * G] = x.reshape(n, G, *to.shape[2:])
        return out.cpu().numpy(), lse.cpu().numpy(), tuple(x.cpu().numpy() for x in (mass, qk, seen, vmax))

    def plan(self, **bounds):
        d, kv = self.descs(**bounds)
        main, *join = hq.hq_attn_plan(d, kv, len(self.new), self.total, self.prefix)
        return {**{k: int(v) for k, v in re.findall(r"(\w+)=(\d+)", main)}, "join": len(join), "kernel": main.split(" ")[0]}

    def planned(self, bounds=None, **want):
        """Asserts a field to be a number, or to be at least that of a tuple of one."""
        p = self.plan(**(bounds or {}))
        for k, v in want.items():
            assert p[k] >= v[0] if isinstance(v, tuple) else p[k] == v, (k, v, p)
        return self


def test_the_reference_is_the_definition():
    """The oracle on the card and the one that goes key by key agree."""
    note("attn reference")
    for c in (Case([40, 3, 70], [3, 5, 20], 4, 2, 16, "fp16", prefix=9, softcap=2.0, seed=1), Case([2, 0, 5], [5, 3, 1], 4, 1, 32, "bf16", "fp8", seed=2)):
        a, b = c.oracle(), AttnCase.oracle(c)
        for x, y in zip((a[0], a[1], *a[2]), (b[0], b[1], *b[2])):
            fin = np.isfinite(y)
            assert np.array_equal(fin, np.isfinite(x)) and np.abs(x[fin] - y[fin]).max() < 1e-12


# lengths and new tokens: single tokens and drafts; a prompt chunk among them
FEW, MANY = ([1700, 77, 2001], [1, 2, 1]), ([1300, 400], [200, 90])
CUT_FEW, CUT_MANY = dict(joint=0, prefix=(2,), few=(2,), many=0, join=1), dict(joint=0, prefix=(2,), many=(2,), join=1)


@pytest.mark.parametrize("block", [1, 3, 8, 24, 64, 200])
@pytest.mark.parametrize("head_major,cache", [(False, "fp16"), (True, "fp16"), (True, "fp8")])
@pytest.mark.parametrize("lens,new,want", [(*FEW, CUT_FEW), (*MANY, CUT_MANY)])
def test_pages_behind_a_prefix_in_parts(block, head_major, cache, lens, new, want):
    """Pages of any size, both orders, with a gap between them, a prefix that ends inside a page."""
    note(f"attn pages {block} {head_major} {cache} {lens}")
    Case(lens, new, 8, 2, 64, "fp16", cache, block=block, prefix=905, head_major=head_major, pad=48, seed=block).planned(**want).check()


@pytest.mark.parametrize("block,head_major", [(24, True), (64, True), (24, False), (200, False)])
def test_pages_of_prompts_alone(block, head_major):
    note(f"attn prompt pages {block}")
    Case([700, 400], [200, 400], 8, 2, 64, "bf16", block=block, head_major=head_major, pad=16, seed=block).planned(prefix=0, many=(2,)).check()
    Case([333, 90], [333, 77], 4, 2, 128, "bf16", "fp8", block=block, head_major=head_major, prefix=40, seed=3).planned(many=(1,)).check()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8"), ("fp16", "fp8")])
@pytest.mark.parametrize("D", [16, 64, 80, 96, 128, 144, 240, 256])
def test_types_and_widths_in_parts(dtype, cache, D):
    note(f"attn widths {dtype} {cache} {D}")
    Case([1500, 40, 700], [1, 2, 9], 8, 2, D, dtype, cache, prefix=700, seed=D).planned(**CUT_FEW).check()
    Case([1500, 40, 700], [1, 2, 70], 8, 2, D, dtype, cache, prefix=700, seed=D).planned(**CUT_MANY).check()


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 1), (12, 12), (33, 1), (28, 4), (64, 2), (64, 1)])
def test_head_layouts_in_parts(Hq, Hk):
    note(f"attn heads {Hq}/{Hk}")
    Case([1537, 200, 1065], [1, 3, 1], Hq, Hk, 64, "fp16", prefix=1333, seed=Hq).planned(joint=0, prefix=(2,), join=1).check()


@pytest.mark.parametrize("cache", ["fp16", "fp8"])
@pytest.mark.parametrize("softcap", [2.0, 30.0, 500.0])
@pytest.mark.parametrize("lens,new,want", [(*FEW, CUT_FEW), (*MANY, CUT_MANY)])
def test_caps_in_parts(softcap, cache, lens, new, want):
    note(f"attn caps {softcap} {cache} {lens}")
    c = Case(lens, new, 8, 4, 64, "fp16", cache, prefix=900, softcap=softcap, q_gain=3.0, seed=2).planned(**want)
    assert c.plan()["kernel"].endswith(",wide>") == (softcap > 64)
    c.check()


@pytest.mark.parametrize("lens,new,prefix,want", [(*FEW, 900, CUT_FEW), (*MANY, 905, CUT_MANY), ([5000], [1], 0, dict(few=(2,), join=1))])
def test_padding_rows_are_not_written_by_a_join(lens, new, prefix, want):
    note(f"attn padding rows {lens} {prefix}")
    n = sum(new)
    c = Case(lens, new, 8, 2, 64, "bf16", prefix=prefix, seed=9, total_rows=n + 7, q_pad=16).planned(**want)
    got, ls, args = c.check()
    assert (got[n:] == 7).all() and (ls[n:] == 7).all()
    assert (args[14][:, 8 * 64:] == 7).all()


@pytest.mark.parametrize("lens,new,prefix,want", [(*FEW, 900, CUT_FEW), (*MANY, 905, CUT_MANY)])
def test_joins_on_another_stream_and_without_lse(lens, new, prefix, want):
    note(f"attn other stream {lens}")
    c = Case(lens, new, 8, 2, 64, "bf16", prefix=prefix, seed=9).planned(**want)
    first, _, _ = c.run()
    got, _, _ = c.run(stream=torch.cuda.Stream(), lse=False)
    assert np.array_equal(got, first)


# ---------------------------------------------------------------------------
# what is not finite
# ---------------------------------------------------------------------------

def raw(c, side):
    return c.store[side].view(torch.uint8) if c.cache == "fp8" else c.store[side].view(torch.int16)


def spoil(c, side, r, i, h, d):
    """NaN into element d of head h of the own key i of request r."""
    raw(c, side)[int(c.table[r, i // c.block]), i % c.block, h, d] = 0x7F if c.cache == "fp8" else 0x7FC0 if c.dtype == "bf16" else 0x7E00


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,new,prefix,want", [([1500, 900], [15, 12], 600, CUT_FEW), ([1500, 900], [15, 12], 0, dict(few=(2,), many=0, join=1)),
                                                  ([600, 41], [16, 9], 0, dict(few=1, many=0, join=0)), (*MANY, 905, CUT_MANY),
                                                  ([1300], [200], 0, dict(many=(2,), join=1))])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(cache, lens, new, prefix, want):
    """NaN in V at new tokens in every stripe of 32 keys that the waves take turns with, in whichever
    part they lie, in K at one, and everywhere beyond the lengths."""
    note(f"attn not finite {cache} {lens} prefix {prefix}")
    c = Case(lens, new, 8, 2, 64, "bf16", cache, prefix=prefix, seed=4).planned(**want)
    clean, _, _ = c.run()
    held = torch.zeros(c.nb, c.block, dtype=torch.bool)
    for i in range(prefix):
        held[int(c.prefix_ids[i // c.block]), i % c.block] = True
    for r, n in enumerate(lens):
        for i in range(n):
            held[int(c.table[r, i // c.block]), i % c.block] = True
    for side in range(2):
        raw(c, side)[~held] = 0x7F if cache == "fp8" else 0x7FC0
    got, _, _ = c.run()
    assert np.array_equal(got, clean)
    expect = clean.copy()
    for r, (n, m) in enumerate(zip(lens, new)):
        t0 = int(c.cu[r])
        for j, at in enumerate(range(0, m, 1 if m < 32 else 13)):  # the at-th new token
            d = j % 60
            spoil(c, 1, r, n - m + at, j % 2, d)
            expect[t0 + at:t0 + m, 4 * (j % 2):4 * (j % 2) + 4, d] = np.nan
    r, at = len(new) - 1, new[-1] // 2
    spoil(c, 0, r, lens[r] - new[r] + at, 1, 5)
    expect[int(c.cu[r]) + at:int(c.cu[r + 1]), 4:] = np.nan
    got, _, _ = c.run()
    np.testing.assert_array_equal(got, expect)


# ---------------------------------------------------------------------------
# long and short together, loose bounds
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,new,Hq,Hk,D,want", [
    ([20000, 4000, 900], [1, 4000, 1], 32, 8, 16, dict(few=1, many=1, join=0)),    # long decodes in one part
    ([9000, 700, 4000], [1, 600, 1], 8, 2, 64, dict(few=(2,), many=(2,), join=1)),
    ([20000, 1500], [1, 1500], 8, 1, 32, dict(few=(2,), many=(2,), join=1))])
@pytest.mark.parametrize("exact", [False, True])
def test_a_prompt_chunk_beside_long_decodes(lens, new, Hq, Hk, D, want, exact):
    note(f"attn chunk beside decodes {lens}")
    c = Case(lens, new, Hq, Hk, D, "bf16", seed=5)
    total = sum(lens) if exact else 0
    if not exact:
        c.planned(**want)
    c.check(total_kv=total)


@pytest.mark.parametrize("prefix", [100, 1000])
def test_prompts_that_walk_the_prefix_themselves(prefix):
    """Several requests whose rows fill 16 tiles each: no product for all."""
    note(f"attn prompts walk {prefix}")
    Case([600, 500], [600, 500], 8, 1, 64, "bf16", prefix=prefix, seed=6).planned(joint=1, many=(2,)).check()
    Case([700, 530], [700, 530], 8, 1, 64, "fp16", "fp8", prefix=prefix + 5, block=24, seed=6).planned(joint=1).check()


@pytest.mark.parametrize("prefix,lens,joint,parts", [(1030, [20, 2, 9], 0, 1), (1030, [900, 1100, 1000], 0, 1), (129, [3, 1, 20], 1, 1), (1030, [300], 1, 2)])
def test_both_ways_of_a_prefix(prefix, lens, joint, parts):
    note(f"attn prefix {prefix} {lens}")
    c = Case(lens, [1] * len(lens), 8, 2, 128, "bf16", prefix=prefix, seed=prefix)
    c.planned(joint=joint, few=(parts,), prefix=0 if joint else (1,), join=int(not joint or parts > 1)).check()


@pytest.mark.parametrize("lens,new,prefix", [([300, 700], [1, 2], 0), ([4000] * 5, [1, 0, 1, 1, 1], 0), ([700, 30, 5], [90, 1, 2], 300)])
def test_bounds_of_a_captured_graph(lens, new, prefix):
    """The largest context and no sum of the lengths: longer parts, the same values."""
    note(f"attn loose {lens} prefix {prefix}")
    c = Case(lens, new, 8, 2, 64, "bf16", prefix=prefix, seed=9)
    for bounds in (dict(max_kv=131072), dict(max_kv=131072, max_new=2 * max(new)), dict(max_kv=131072, total_kv=sum(lens))):
        c.check(**bounds)
