"""The prompt-side operators together, checked against what stands in the cache: each row is compared with the formula when it is
written, and every later attention, over forked, copied, trimmed and compacted pages, with dense attention over the rows as
they were stored. With FP8 the bound is then that of the arithmetic alone, so that rows from a wrong page do not pass."""
import math

import pytest
import torch

from paged_kv_speculative_gb300 import pa_verify as pv
from .test_prefill_flow import D, HKV, HQ, PAGE, Server

pytestmark = pytest.mark.gpu


class Stored(Server):
    def rows(self, b, at):
        """(k, v, v's scale) of tokens ``at`` of row b, in 64 bits, and K's scale."""
        page, off = self.table[b, at // PAGE].long(), at % PAGE
        out = []
        for c, s in ((self.k, self.ks), (self.v, self.vs)):
            x = c[page, :, off]
            x = x.double() if s is None else x.view(torch.float8_e4m3fn).double() * s[page, :, off].double()[..., None]
            out.append((x, None if s is None else s[page, :, off].double()))
        return out

    def stored(self, b, n):
        """The last n rows of b's history, new ones as the formula has them, become what the cache holds."""
        new = [i for i in range(len(self.history[b]) - n, len(self.history[b])) if len(self.history[b][i]) == 2]
        if not new:
            return
        (k, ks), (v, vs) = self.rows(b, torch.tensor(new, device="cuda"))
        for w, (got, s) in enumerate(((k, ks), (v, vs))):
            want = torch.stack([self.history[b][i][w] for i in new])
            # rotated in fp32: within 2^-18 of the row's largest; then half a step of bf16 (2^-8) or of E4M3 (2^-4, and 2^-10 of the scale)
            eps = want.abs().amax(-1, keepdim=True) * 2.0 ** -18
            half = want.abs() * 2.0 ** -8 if s is None else want.abs() * 2.0 ** -4 * 1.01 + s[..., None] * 2.0 ** -10 * 1.01
            assert ((got - want).abs() <= half + eps).all()
        for j, i in enumerate(new):
            self.history[b][i] = (k[j], v[j], torch.ones_like(v[j, :, 0]) if vs is None else vs[j])

    def check(self, q, out, ql, verify=False):
        """Against the stored rows: the output's half step (2^-8), that of P (2^-8) and, FP8, of V (2^-8), of sum p |v|; FP8 keys
        in f16 (2^-11 an entry, 2^-10 of a score's sum of sizes on a weight); fp32 2^-12. The verify kernel's FP8 weights are two
        E4M3 terms: 2^-6, and 2^-9 of the largest weight times scale for every code."""
        i, fp8 = 0, self.kv == pv.KV_FP8_E4M3
        for b, n in enumerate(ql):
            if not n:
                continue
            self.stored(b, n)
            k, v = (torch.stack([h[w] for h in self.history[b]]).repeat_interleave(HQ // HKV, 1) for w in range(2))
            sv = torch.stack([h[2] for h in self.history[b]]).repeat_interleave(HQ // HKV, 1)  # [L, HQ]
            L, x = k.shape[0], q[i:i + n].double()
            s = torch.einsum("ihd,thd->hit", x, k) / math.sqrt(D)
            seen = torch.arange(L, device="cuda") <= L - n + torch.arange(n, device="cuda")[:, None]
            p = s.masked_fill(~seen, -math.inf).softmax(-1)
            want, size = torch.einsum("hit,thd->ihd", p, v), torch.einsum("hit,thd->ihd", p, v.abs())
            share, floor = 2.0 ** -8 + 2.0 ** -12, 0.0
            if fp8:
                spread = (torch.einsum("ihd,thd->hit", x.abs(), k.abs()) / math.sqrt(D)).amax(-1).t()[..., None]
                share = (2.0 ** -6 if verify else 2.0 ** -7) + 2.0 ** -11 + spread * 2.0 ** -10
                if verify:
                    codes = torch.einsum("it,thd->ihd", seen.double(), v.abs() / sv[..., None])
                    floor = (p * sv.t()[:, None]).amax(-1).t()[..., None] * codes * 2.0 ** -9
            assert ((out[i:i + n].double() - want).abs() <= want.abs() * 2.0 ** -8 + share * size + floor).all(), f"row {b}"
            i += n

    def attend(self, ql, verify=False):
        """The last ql[b] tokens of the rows attend once more, with queries of their own."""
        q = torch.randn((sum(ql), HQ, D), device="cuda", generator=self.gen).to(torch.bfloat16)
        dev, lens = torch.tensor(ql, dtype=torch.int32, device="cuda"), self.lens.tolist()
        if verify:
            live = [b for b, n in enumerate(ql) if n]
            va = pv.VerifyAttention(HQ, HKV, D, self.kv, self.k.shape[0], self.table.shape[1], [lens[b] for b in live], [ql[b] for b in live])
            return q, va(q, self.k, self.v, self.ks, self.vs, self.table[live], self.lens[live], dev[live], 1 / math.sqrt(D)), ql
        return q, self.chunk(q, self.k, self.v, self.ks, self.vs, self.table, self.lens, dev, 1 / math.sqrt(D)), ql

    def step(self, ql):
        """Server.step's first check is chunk attention's, its second verify attention's."""
        kinds = iter((False, True))
        self.check = lambda q, out, ql: Stored.check(self, q, out, ql, verify=next(kinds))
        super().step(ql)
        del self.check


def flow(kv):
    s = Stored(kv)
    s.step([200, 37, 0, 0, 0, 0])
    s.step([133, 1, 0, 5, 0, 0])
    s.pool.fork(*s.tables(), *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 0, 1], [2, 4, 5])))
    for p, c in ((0, 2), (0, 4), (1, 5)):
        s.history[c] = list(s.history[p])
    s.step([6, 6, 6, 0, 6, 6])
    s.step([1, 30, 2, 1, 0, 64])
    s.resize([-1, 20, 0, -1, -1, 90])
    table, ref, src, dst, moves = s.pool.compact(*s.tables(), in_place=True)
    s.pool.copy(src, dst, moves)
    s.step([8, 3, 0, 2, 8, 1])
    s.step([70, 0, 90, 17, 1, 0])
    return s


@pytest.mark.parametrize("kv", [pv.KV_BF16, pv.KV_FP8_E4M3])
def test_stored_rows_through_branches_drafts_and_compaction(kv):
    s = flow(kv)
    lens = s.lens.tolist()
    s.check(*s.attend([min(50, n) for n in lens]))
    s.check(*s.attend([min(8, n) for n in lens]))
    s.check(*s.attend([min(8, n) for n in lens], verify=True), verify=True)
    assert s.pool.device_errors() == 0 and s.chunk.device_errors() == 0


@pytest.mark.parametrize("kv", [pv.KV_BF16, pv.KV_FP8_E4M3])
@pytest.mark.parametrize("verify", [False, True])
def test_the_check_sees_a_wrong_page(kv, verify):
    """The same answers against a history in which one page is another sequence's: they do not pass."""
    s = flow(kv)
    lens, b, other = s.lens.tolist(), 0, 2
    assert lens[b] > 300 and lens[other] >= 48
    for at in (0, 160, lens[b] // PAGE * PAGE - PAGE):
        got = s.attend([8, 0, 0, 0, 0, 0], verify)
        s.check(*got, verify=verify)
        right = s.history[b]
        s.history[b] = right[:at] + s.history[other][16:32] + right[at + PAGE:]
        with pytest.raises(AssertionError, match="row 0"):
            s.check(*got, verify=verify)
        s.history[b] = right
