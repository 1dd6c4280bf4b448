"""Calls of the decoder-layer operators that their documentation allows: several
at once on streams of their own, and operands that lie far apart (offsets past
2^31 elements and 2^32 bytes).  The same arithmetic runs in the same order, so
results equal those of a dense call alone bit for bit."""
import pytest
import torch

from megatron_tensor_transformer_logical_b200 import binding as L
from tests.parity import need_gpu

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    L.tp_device_status()


class Job:
    """One training or decoding chain on its own buffers."""

    def __init__(self, seed, s, heads, kv, d, f, window, sinks, dt):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *sh, std=1.0: (torch.randn(*sh, generator=self.g, device="cuda") * std).to(dt)
        e = lambda *sh, t=dt: torch.empty(*sh, dtype=t, device="cuda")
        h = heads * d
        self.cfg = (s, heads, kv, d, f, window, sinks, h)
        self.Q, self.K, self.V, self.dO = rn(s, h), rn(s, kv * d), rn(s, kv * d), rn(s, h)
        self.gq, self.gk = rn(d), rn(d)
        self.pos = torch.arange(s, dtype=torch.int32, device="cuda")
        self.fr = torch.pow(10000.0, -torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2
                            / d)
        self.lens = torch.full((1,), s, dtype=torch.int32, device="cuda")
        self.out = dict(Qr=e(s, h), Kr=e(s, kv * d), O=e(s, h), LSE=e(1, heads, s, t=torch.float32),
                        dQr=e(s, h), dKr=e(s, kv * d), dV=e(s, kv * d), dQ=e(s, h), dK=e(s, kv * d),
                        dgq=e(d), dgk=e(d), O1=e(1, h))
        self.ws = (L.window_attn_workspace(1, s, s, heads, kv, d, window, sinks),
                   L.qk_norm_rope_workspace(s, d),
                   L.window_attn_decode_workspace(1, s, heads, kv, d, window, sinks))
        self.glu = dt == BF
        if self.glu:
            self.Wgu, self.Wd = rn(h, 2 * f, std=h ** -0.5), rn(f, h, std=f ** -0.5)
            self.out.update(Z=e(s, h), Z1=e(1, h), dX=e(s, h), dWgu=e(h, 2 * f), dWd=e(f, h))
            w = lambda op: L.workspace(op, s, h, f, 0, 1, L.TP_BF16)
            self.wsg = (w(L.TP_OP_GLU_FWD), w(L.TP_OP_GLU_BWD))

    def run(self):
        s, heads, kv, d, f, W, S, h = self.cfg
        o = self.out
        L.tp_qk_norm_rope_fwd(self.Q, self.K, self.gq, self.gk, self.pos, self.fr, o["Qr"], o["Kr"],
                              d)
        L.tp_window_attn_fwd(o["Qr"], o["Kr"], self.V, o["O"], o["LSE"], 1, heads, kv, W, S)
        L.tp_window_attn_bwd(o["Qr"], o["Kr"], self.V, o["O"], o["LSE"], self.dO, o["dQr"],
                             o["dKr"], o["dV"], 1, heads, kv, W, S, self.ws[0])
        L.tp_qk_norm_rope_bwd(self.Q, self.K, self.gq, self.gk, self.pos, self.fr, o["dQr"],
                              o["dKr"], o["dQ"], o["dK"], o["dgq"], o["dgk"], d, self.ws[1])
        L.tp_window_attn_decode(o["Qr"][-1:], o["Kr"][None], self.V[None], self.lens, o["O1"], None,
                                heads, kv, W, S, self.ws[2])
        if self.glu:
            L.tp_glu_fwd(o["O"], self.Wgu, None, self.Wd, None, o["Z"], None, 1, 0, self.wsg[0])
            L.tp_glu_fwd(o["O1"], self.Wgu, None, self.Wd, None, o["Z1"], None, 1, 0, self.wsg[0])
            L.tp_glu_bwd(o["O"], self.Wgu, None, self.Wd, None, self.dO, o["dX"], o["dWgu"], None,
                         o["dWd"], None, 1, 0, self.wsg[1])


def test_chains_on_streams_of_their_own():
    jobs = [Job(0, 700, 8, 2, 64, 1024, 100, 4, BF), Job(1, 333, 4, 1, 128, 512, 400, 0, BF),
            Job(2, 900, 12, 3, 64, 0, 257, 2, FP), Job(3, 20, 16, 4, 128, 2816, 8, 1, BF)]
    refs = []
    for j in jobs:
        j.run()
        torch.cuda.synchronize()
        refs.append({n: v.clone() for n, v in j.out.items()})
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        for j in jobs:
            for v in j.out.values():
                v.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(4):
            for j, st in zip(jobs, streams):
                with torch.cuda.stream(st):
                    j.run()
        torch.cuda.synchronize()
        for j, ref in zip(jobs, refs):
            for n in ref:
                assert torch.equal(j.out[n], ref[n]), (j.cfg, n)


@pytest.fixture(scope="module")
def far():
    """Rows 2^24 + 8 elements apart, 140 of them: past 2^31 elements from row 128 on."""
    need_gpu()
    buf = torch.empty(140 * ((1 << 24) + 8), dtype=BF, device="cuda")
    yield buf
    del buf
    torch.cuda.empty_cache()


def spread(buf, first, *tensors):
    """Copies of [rows, cols] tensors as columns of the far rows, from `first` on."""
    out, ld = [], (1 << 24) + 8
    for t in tensors:
        v = torch.as_strided(buf, t.shape, (ld, 1), first)
        v.copy_(t)
        out.append(v)
        first += t.shape[1]
    return out


def test_far_rows(far):
    s, heads, kv, d, W, S = 140, 4, 2, 64, 50, 3
    j = Job(5, s, heads, kv, d, 64, W, S, BF)
    j.run()
    o = j.out
    names = ("Qr", "Kr", "O", "dQr", "dKr", "dV", "dQ", "dK")
    Q, K, V, dO, *outs = spread(far, 0, j.Q, j.K, j.V, j.dO, *(o[n] for n in names))
    q = dict(zip(names, outs))
    for v in outs:
        v.fill_(float("nan"))
    lse, dgq, dgk = torch.empty_like(o["LSE"]), torch.empty_like(o["dgq"]), torch.empty_like(o["dgk"])
    L.tp_qk_norm_rope_fwd(Q, K, j.gq, j.gk, j.pos, j.fr, q["Qr"], q["Kr"], d)
    L.tp_window_attn_fwd(q["Qr"], q["Kr"], V, q["O"], lse, 1, heads, kv, W, S)
    L.tp_window_attn_bwd(q["Qr"], q["Kr"], V, q["O"], lse, dO, q["dQr"], q["dKr"], q["dV"], 1,
                         heads, kv, W, S, j.ws[0])
    L.tp_qk_norm_rope_bwd(Q, K, j.gq, j.gk, j.pos, j.fr, q["dQr"], q["dKr"], q["dQ"], q["dK"], dgq,
                          dgk, d, j.ws[1])
    for n in names:
        assert torch.equal(q[n], o[n]), n
    assert torch.equal(lse, o["LSE"]) and torch.equal(dgq, o["dgq"]) and torch.equal(dgk, o["dgk"])


def test_decode_over_a_far_cache(far):
    """Sequences 2^30 elements apart, or keys 2^24: the last ones past 2^31."""
    b, heads, kv, d = 3, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    rn = lambda *sh: torch.randn(*sh, generator=g, device="cuda").to(BF)
    for cap, strides in ((300, (1 << 30, 2 * kv * d, 1)), (130, (1024, (1 << 24) + 8, 1))):
        Q, K, V = rn(b, heads * d), rn(b, cap, kv * d), rn(b, cap, kv * d)
        lens = torch.tensor([cap, 1, cap - 1], dtype=torch.int32, device="cuda")
        ws = L.window_attn_decode_workspace(b, cap, heads, kv, d, cap, 0)
        O, O2 = torch.empty_like(Q), torch.empty_like(Q)
        L.tp_window_attn_decode(Q, K, V, lens, O, None, heads, kv, cap, 0, ws)
        fk, fv = (torch.as_strided(far, K.shape, strides, first) for first in (0, kv * d))
        fk.copy_(K)
        fv.copy_(V)
        L.tp_window_attn_decode(Q, fk, fv, lens, O2, None, heads, kv, cap, 0, ws)
        assert torch.equal(O, O2), cap
