"""The four entry points together, as a server uses them: prompts, decoding steps, drafted tokens,
a request that ends and one that takes its pages, every step's attention against the binary64
statement over everything stored so far; and decoding steps captured once and replayed."""
import numpy as np
import pytest
import torch

from tests import kv_common as kc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def omq(cuda_device):
    from post_quantization_lwc_b200 import build
    build.build()
    from post_quantization_lwc_b200 import omq as m
    return m


class Server:
    def __init__(self, omq, dev, n_req, n_pages, Hkv, G, D, page, abits, max_len=512):
        self.omq, self.dev, self.abits = omq, dev, abits
        self.Hkv, self.G, self.D, self.page = Hkv, G, D, page
        self.cache = omq.KVCache(n_req, n_pages, Hkv, D, page=page, max_len=max_len, device=dev)
        self.gen = torch.Generator().manual_seed(n_req + D)
        r = lambda *s: torch.randn(*s, generator=self.gen)  # noqa: E731
        self.sa, self.so, self.dl = torch.exp(0.3 * r(Hkv, D)), torch.exp(0.3 * r(Hkv, D)), 0.2 * r(Hkv, D)
        self.rope = self.cache.rope.cpu().numpy()
        self.seen = [dict(k=[], v=[]) for _ in range(n_req)]      # encoded rows per request

    def qkv(self, rows):
        n = (self.Hkv * self.G + 2 * self.Hkv) * self.D
        return torch.randn(rows, n, generator=self.gen)

    def split(self, x):
        a, b, d = self.Hkv * self.G, self.Hkv, self.D
        cut = lambda i, n: x[:, i * d:(i + n) * d].unflatten(1, (n, d))  # noqa: E731
        return cut(0, a), cut(a, b), cut(a + b, b)

    def device_step(self, new, x, max_q):
        step = self.cache.plan(new, x.shape[0])
        q, k, v = self.split(x)
        qt = self.cache.append(step, k, v, q, s_a=self.sa.to(self.dev), s_o=self.so.to(self.dev),
                               delta_o=self.dl.to(self.dev), abits=self.abits)
        return step, qt, self.cache.attend(step, qt, max_q)

    def note(self, step, x):
        """Appends the step's rows to the statement's own record, from the step's maps."""
        q, k, v = (t.float().numpy() for t in self.split(x))
        pos, req = step["positions"].cpu().numpy(), step["requests"].cpu().numpy()
        live = req >= 0
        cos, sin = self.rope[0][np.maximum(pos, 0)], self.rope[1][np.maximum(pos, 0)]
        k = (kc.rotate(k, cos, sin) * self.sa.numpy()).astype(np.float32)
        v = ((v - self.dl.numpy()).astype(np.float32) / self.so.numpy()).astype(np.float32)
        for t in np.nonzero(live)[0]:
            mine = self.seen[req[t]]
            assert len(mine["k"]) == pos[t]
            mine["k"].append(kc.encode(k[t]))
            mine["v"].append(kc.encode(v[t]))

    def check(self, step, qt, out, every=1):
        pos, req = step["positions"].cpu().numpy(), step["requests"].cpu().numpy()
        got, q = out.double().cpu().numpy(), qt.double().cpu().numpy()
        for t in np.nonzero(req >= 0)[0][::every]:
            mine = self.seen[req[t]]
            step = 2.0 ** -11 if (req == req[t]).sum() * self.G > 32 else 0.0   # float16 operands
            k, v = ([np.stack([r[i] for r in mine[n][:pos[t] + 1]]) for i in range(3)] for n in ("k", "v"))
            for h in range(0, self.Hkv * self.G, 3):
                j = h // self.G
                o, _, tol, _ = kc.attend(q[t, h], *(a[:, j] for a in k), *(a[:, j] for a in v),
                                         np.ones(pos[t] + 1, bool), self.D ** -0.5, 2.0 ** -11, step)
                assert np.all(np.abs(got[t, h] - o) <= tol), (t, h)


@pytest.mark.parametrize("Hkv,G,D,page,abits", [(2, 4, 128, 16, 16), (3, 1, 64, 32, 4)])
def test_serving_steps(omq, cuda_device, Hkv, G, D, page, abits):
    s = Server(omq, cuda_device, 3, 200 // page + 2, Hkv, G, D, page, abits)
    rounds = [  # new tokens per request, what each is granted
        ([40, 0, 17], [40, 0, 17]),          # two prompts
        ([1, 33, 1], [1, 33, 1]),            # decoding beside a prompt
        ([5, 5, 5], [5, 5, 5]),              # drafted tokens
        ([1, 1, 1], [1, 1, 1]),
        ([-1, 2, 400], [0, 2, 0]),           # one ends; one asks for more than the pool holds
        ([50, 1, 1], [50, 1, 1]),            # a new request in its place, on its pages
        ([1, 1, 1], [1, 1, 1]),
    ]
    for new, want in rounds:
        for b, n in enumerate(new):
            if n < 0:
                s.seen[b] = dict(k=[], v=[])
        x = s.qkv(max(1, sum(n for n in new if n > 0)))
        step, qt, out = s.device_step(torch.tensor(new, dtype=torch.int32, device=cuda_device),
                                      x.to(cuda_device), max(1, max(new)))
        omq.sync_check()
        cu = step["cu"].cpu().numpy()
        assert np.array_equal(np.diff(cu), want)
        s.note(step, x)
        s.check(step, qt, out, every=1 if len(x) < 20 else 7)
        assert np.array_equal(s.cache.lens.cpu().numpy(), [len(r["k"]) for r in s.seen])


def test_captured_decoding_steps(omq, cuda_device):
    """One decoding step captured, replayed over a page's end, against eager steps of a second
    cache bit for bit; its rows are padded beyond the live requests."""
    dev = cuda_device
    a = Server(omq, dev, 4, 40, 2, 4, 128, 16, 16)
    b = Server(omq, dev, 4, 40, 2, 4, 128, 16, 16)
    prompt = torch.tensor([13, 30, 0, 64], dtype=torch.int32, device=dev)
    x = a.qkv(107).to(dev)
    for s in (a, b):
        s.scales = [t.to(dev) for t in (s.sa, s.so, s.dl)]
        s.device_step(prompt, x, 64)
    new, xin = torch.zeros(4, dtype=torch.int32, device=dev), torch.zeros_like(a.qkv(6).to(dev))

    def decode(s):
        step = s.cache.plan(new, 6)                     # six rows, at most four in use
        q, k, v = s.split(xin)
        sa, so, dl = s.scales
        qt = s.cache.append(step, k, v, q, s_a=sa, s_o=so, delta_o=dl)
        return step, s.cache.attend(step, qt, 1)

    decode(a), decode(b)                                # warm-up: no request takes a token
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_a, out_a = decode(a)
    for i in range(20):
        new.copy_(torch.tensor([1, 1, i % 2, -1 if i == 9 else 1 if i < 9 else 0], dtype=torch.int32))
        xin.copy_(a.qkv(6))
        graph.replay()
        step_b, out_b = decode(b)
        n = int(step_b["cu"][-1])
        for key in step_a:
            assert torch.equal(step_a[key], step_b[key]), (i, key)
        assert torch.equal(out_a[:n], out_b[:n]), i
        assert torch.equal(a.cache.table, b.cache.table)
    omq.sync_check()


def test_a_whole_step_on_a_side_stream(omq, cuda_device):
    """plan, append, read and attend with stream=, and the rotary table made there, give what
    they give on the current stream; a stream of no device that fits is refused."""
    side, got = torch.cuda.Stream(), []
    for stream in (None, side):
        s = Server(omq, cuda_device, 3, 60, 2, 2, 64, 16, 16)
        rope = omq.rope_table(512, 64, device="cuda", stream=stream)
        x = [s.qkv(40).to(cuda_device).half() for _ in range(2)]
        torch.cuda.synchronize()
        for new, rows in zip(([20, 0, 17], [1, 3, 1]), x):
            new = torch.tensor(new, dtype=torch.int32, device=cuda_device)
            torch.cuda.synchronize()
            step = s.cache.plan(new, rows.shape[0], stream=stream)
            q, k, v = s.split(rows)
            qt = torch.zeros(40, 4, 64, dtype=torch.float16, device=cuda_device)
            torch.cuda.synchronize()
            s.cache.append(step, k, v, q, q_out=qt, stream=stream)
            out = torch.zeros_like(qt)
            torch.cuda.synchronize()
            s.cache.attend(step, qt, 20, out=out, stream=stream)
            kk, vv = omq.kv_read(s.cache.pool, step["slots"], stream=stream)
            torch.cuda.synchronize()
            got.append([rope, step["slots"].clone(), qt, out, kk, vv, s.cache.lens.clone()])
    omq.sync_check()
    for a, b in zip(got[:2], got[2:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(ValueError):
        omq.rope_table(8, 64, device="cpu", stream=side)
