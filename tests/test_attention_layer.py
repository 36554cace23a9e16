"""GPU tests of an attention layer as it is served: the QKV product, the append
to the cache, the attention and the output product handing each other their
device buffers, eagerly, on other streams and from replayed graphs."""
import numpy as np
import pytest

import attention_ref as ref
import block_scaled_precision_mxfp4_amd as mx
import experts_ref
import oracle
from test_attention import E4M3, Batch, bf16, check, check_append, dev, say, workspace

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mxgpu import assert_parity, dev_bf16, dev_u8, host_bits  # noqa: E402


class Layer:
    """hidden -> (quantize, QKV product, append, attention, output product) -> hidden."""

    def __init__(self, new, lens, H, Hk, D, hidden, page, fp8, seed, rows=None):
        rng = np.random.default_rng(seed)
        self.b = b = Batch(rng, new, lens, Hk, D, page, fp8)
        if fp8:
            b.k_scale = b.v_scale = np.full(Hk, 1 / 16, np.float32)
        self.cache = b.cache()
        self.T = b.T if rows is None else rows
        self.H, self.D, self.hidden, self.N = H, D, hidden, (H + 2 * Hk) * D
        T = self.T
        self.w = [self.weight(rng, self.N, hidden), self.weight(rng, hidden, H * D)]
        self.wd = [tuple(dev_u8(x) for x in w) for w in self.w]
        self.freq = mx.mxgemm_rope_frequencies(D)
        self.freqd = dev(np.asarray(self.freq))
        z = lambda *s, t=torch.uint8: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        self.X, self.A, self.SA = z(T, hidden, t=torch.bfloat16), z(T, hidden // 2), z(T, hidden // 32)
        self.qkv, self.O, self.lse = z(T, self.N, t=torch.bfloat16), z(T, H * D, t=torch.bfloat16), z(T, H, t=torch.float32)
        self.B, self.SB, self.Y = z(T, H * D // 2), z(T, H * D // 32), z(T, hidden, t=torch.bfloat16)
        self.ws = workspace(T, b.S, H, Hk, D)

    @staticmethod
    def weight(rng, N, K):
        return rng.integers(0, 256, (N, K // 2), dtype=np.uint8), rng.integers(120, 124, (N, K // 32), dtype=np.uint8)

    def feed(self, seed):
        rng = np.random.default_rng(seed)
        self.X.copy_(dev_bf16(bf16(rng, self.T, self.hidden)))
        self.b.k.copy_(dev(self.b.kc if self.b.fp8 else self.b.kc.view(np.int16)))
        self.b.v.copy_(dev(self.b.vc if self.b.fp8 else self.b.vc.view(np.int16)))

    def run(self, stream=None):
        T, H, Hk, D = self.T, self.H, self.b.kv_heads, self.D
        s = stream.cuda_stream if stream is not None else None
        mx.mxgemm_quantize(self.A, self.SA, self.X, T, self.hidden, stream=s)
        mx.mxgemm_run_noalloc(self.qkv, None, self.A, self.wd[0][0], self.SA, self.wd[0][1], 1.0, 0.0, T, self.N, self.hidden, stream=s)
        q, k, v = self.qkv, self.qkv[:, H * D:], self.qkv[:, (H + Hk) * D:]
        mx.mxgemm_kv_append(self.cache, T, Q=q, Q_out=q, K=k, V=v, heads=H, ldq=self.N, ldqo=self.N, ldk=self.N, ldv=self.N,
                            freq=self.freqd, rot_dim=D, stream=s)
        mx.mxgemm_paged_attention(self.cache, T, q, self.O, heads=H, scale=D ** -0.5, lse=self.lse, ldq=self.N, ldo=H * D,
                                  A=self.B, scaleA=self.SB, lda=H * D, ldsa=H * D // 32, workspace=self.ws,
                                  workspace_bytes=self.ws.numel(), stream=s)
        mx.mxgemm_run_noalloc(self.Y, None, self.B, self.wd[1][0], self.SB, self.wd[1][1], 1.0, 0.0, T, self.hidden, H * D, stream=s)

    def outputs(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.Y, self.O, self.lse, self.qkv, self.B, self.SB, self.b.k, self.b.v)]

    def forget(self):
        for t in (self.A, self.SA, self.qkv, self.O, self.lse, self.B, self.SB, self.Y):
            t.zero_()

    def check(self):
        """Each stage against the reference from what the stage before it left."""
        torch.cuda.synchronize()
        b, T, H, Hk, D = self.b, self.T, self.H, self.b.kv_heads, self.D
        a, sa = self.A.cpu().numpy(), self.SA.cpu().numpy()
        out, mag = oracle.mxgemm(a, sa, *self.w[0], self.hidden)[:2]
        bits = host_bits(self.qkv)
        assert_parity(bits[:, H * D:], out[:, H * D:], mag[:, H * D:], "QKV")
        # the append: of the product's rows, which its Q has taken the place of
        x = dev_bf16(np.zeros((T, self.N), np.uint16))
        mx.mxgemm_run_noalloc(x, None, self.A, self.wd[0][0], self.SA, self.wd[0][1], 1.0, 0.0, T, self.N, self.hidden)
        rows = host_bits(x)
        q, k, v = (np.ascontiguousarray(rows[:, i * D:j * D]) for i, j in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))
        turned = np.ascontiguousarray(bits[:, :H * D])
        check_append(b, q, k, v, H, turned.reshape(T, H, D), self.freq, D, False, in_place=True, rows=T)
        was = b.kc, b.vc
        b.kc, b.vc = b.pools()
        o = host_bits(self.O)
        live = sum(b.new)
        full = np.full(o.shape, 0x1234, np.uint16)
        full[:live] = o[:live]
        lse = np.full((T, H), 77.0, np.float32)
        lse[:live] = self.lse.cpu().numpy()[:live]
        check(b, turned, H, (full.reshape(T, H, D), lse))
        b.kc, b.vc = was
        want = experts_ref.quantize(o[:live], False)
        assert np.array_equal(self.B.cpu().numpy()[:live], want[0]) and np.array_equal(self.SB.cpu().numpy()[:live], want[1])
        y, mag = oracle.mxgemm(self.B.cpu().numpy(), self.SB.cpu().numpy(), *self.w[1], H * D)[:2]
        assert_parity(host_bits(self.Y), y, mag, "output")


def equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


LAYERS = [  # new, lens, H, Hk, D, hidden, page, fp8, seed
    ([1], [200], 4, 1, 64, 256, 16, False, 1),
    ([1, 1, 1, 1], [1, 700, 33, 64], 8, 2, 128, 256, 16, True, 2),
    ([40, 1, 30], [40, 300, 130], 4, 2, 64, 256, 64, False, 3),
    ([130], [260], 4, 2, 128, 512, 32, True, 4),
]


@pytest.mark.parametrize("case", range(len(LAYERS)))
def test_layer(case):
    a = Layer(*LAYERS[case])
    a.feed(case)
    say("case layer", case)
    a.run()
    a.check()
    first = a.outputs()
    a.feed(case)
    a.run()
    assert equal(first, a.outputs()), "a second run gives other bits"


def test_padded_batch():
    """More rows than the sequences have tokens, as a captured batch of fixed size: the rows behind are left alone."""
    a = Layer([1, 1, 0, 0], [90, 33, 0, 0], 4, 2, 64, 256, 16, False, 5, rows=4)
    a.feed(5)
    a.run()
    a.check()
    assert not a.O[2:].any() and not a.lse[2:].any()


def test_tokens_one_by_one_are_those_of_one_prompt():
    """A prompt appended at once, and token by token: the same cache, and rows within both bounds."""
    rng = np.random.default_rng(6)
    L, H, Hk, D = 40, 4, 2, 64
    b = Batch(rng, [L], [L], Hk, D, 16, False)
    q, k, v = (bf16(rng, L, h * D) for h in (H, Hk, Hk))
    freq = dev(np.asarray(mx.mxgemm_rope_frequencies(D)))
    ws = workspace(L, 1, H, Hk, D)
    caches, rows = [], []
    for step in (L, 1):
        b.cache()
        out = []
        for t in range(0, L, step):
            b.dev[1], b.dev[2] = dev(np.array([0, step], np.int32)), dev(np.array([t + step], np.int32))
            c = b.bind()
            Q, K, V = (dev_bf16(x[t:t + step]) for x in (q, k, v))
            O = torch.zeros_like(Q)
            mx.mxgemm_kv_append(c, step, Q=Q, Q_out=Q, K=K, V=V, heads=H, ldq=H * D, ldqo=H * D, ldk=Hk * D, ldv=Hk * D, freq=freq, rot_dim=D)
            mx.mxgemm_paged_attention(c, step, Q, O, heads=H, scale=D ** -0.5, ldq=H * D, ldo=H * D, workspace=ws, workspace_bytes=ws.numel())
            out.append((host_bits(Q), host_bits(O)))
        caches.append(b.pools())
        rows.append([np.concatenate(x) for x in zip(*out)])
    assert np.array_equal(caches[0][0], caches[1][0]) and np.array_equal(caches[0][1], caches[1][1])
    assert np.array_equal(rows[0][0], rows[1][0])
    b.kc, b.vc = caches[0]
    O, _, off, _ = ref.attention(ref.bf16_to_f64(rows[0][0]).reshape(L, H, D), b.host(), D ** -0.5, True, 0)
    for r in rows:
        assert (np.abs(ref.bf16_to_f64(r[1]).reshape(L, H, D) - O) <= off).all()


def test_layer_on_another_stream():
    a = Layer(*LAYERS[1])
    a.feed(2)
    a.run()
    eager = a.outputs()
    s = torch.cuda.Stream()
    a.feed(2)
    s.wait_stream(torch.cuda.current_stream())
    say("case layer on another stream")
    a.run(stream=s)
    s.synchronize()
    assert equal(eager, a.outputs())


def test_two_attentions_at_once():
    """Two calls on two streams without an order between them, each with its own workspace, read one cache."""
    rng = np.random.default_rng(7)
    b = Batch(rng, [1, 1, 60], [4000, 900, 800], 2, 128, 16, False)
    H, D = 8, 128
    q = [bf16(rng, b.T, H * D) for _ in range(2)]
    cache = b.cache()
    Q = [dev_bf16(x) for x in q]
    O = [torch.zeros_like(x) for x in Q]
    ws = [workspace(b.T, b.S, H, 2, D) for _ in range(2)]

    def call(i, s=None):
        mx.mxgemm_paged_attention(cache, b.T, Q[i], O[i], heads=H, scale=D ** -0.5, ldq=H * D, ldo=H * D, workspace=ws[i],
                                  workspace_bytes=ws[i].numel(), stream=None if s is None else s.cuda_stream)
    want = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        want.append(O[i].clone())
        O[i].zero_()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    say("case two attentions at once")
    for _ in range(10):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(O[i].view(torch.int16), want[i].view(torch.int16))


def test_captured_layers_replay():
    """Two layers captured on their own, one workspace between them, replayed in turn with new inputs, eager work and
    synchronizations between: each replay equals the eager result."""
    layers = [Layer(*LAYERS[1]), Layer(*LAYERS[2])]
    layers[0].ws = layers[1].ws = max((x.ws for x in layers), key=len)
    graphs = []
    for i, a in enumerate(layers):
        a.feed(i)
        a.run()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a.run(stream=s)
        graphs.append(g)
    say("case captured layers")
    for i in range(5):
        want = []
        for a in layers:
            a.feed(20 + i)
            a.run()
            want.append(a.outputs())
        for a in layers:
            a.feed(20 + i)
            a.forget()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for a, w in zip(layers, want):
            assert equal(w, a.outputs()), "replay %d" % i


def test_captured_decode_that_grows():
    """One graph serves every step of a decode: lens, offsets and the inputs change in place, the pages stay."""
    a = Layer([1, 1], [1, 30], 4, 2, 64, 256, 16, False, 9)
    b = a.b
    b.num_pages, b.max_pages = 12, 6
    b.pages = np.random.default_rng(9).permutation(12).astype(np.int32).reshape(2, 6)
    b.kc, b.vc = (bf16(np.random.default_rng(9 + i), 12, 2, 16, 64) for i in range(2))
    a.cache = b.cache()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    a.feed(9)
    a.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        a.run(stream=s)
    say("case captured decode")
    for lens in ([1, 30], [2, 31], [16, 45], [17, 96], [40, 60]):
        b.lens = np.array(lens, np.int32)
        b.dev[2].copy_(dev(b.lens))
        a.feed(lens[0])
        a.forget()
        torch.cuda.synchronize()
        g.replay()
        a.check()


def test_e4m3_codes_of_the_cache_stay_finite():
    """A layer's appended codes are of the cache's scale, no NaN among them."""
    a = Layer(*LAYERS[3])
    a.feed(4)
    a.run()
    torch.cuda.synchronize()
    assert all(np.isfinite(E4M3[x]).all() for x in a.b.pools())
