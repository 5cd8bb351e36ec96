"""The layer operators together with the KDA recurrence, as a serving program runs them:
prompts, then drafts and tokens over shared slots; streams, graphs (needs a B200)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

H, DM = 2, 256          # heads of 128; channels of q, k, v are 3 * H * 128


class KdaLayer:
    """norm -> q, k, v -> short convolution -> KDA -> gated norm of the heads -> output"""

    def __init__(self, slots, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: (torch.randn(*s, generator=g) * s[0] ** -0.5).bfloat16().cuda()  # noqa: E731
        self.qkv, self.gates, self.out = r(DM, 3 * H * 128), r(DM, 2 * H * 128 + H), r(H * 128, DM)
        self.w1, self.w2 = torch.ones(DM).cuda(), torch.ones(128).cuda()
        self.conv = (0.5 * torch.randn(3 * H * 128, 4, generator=g)).cuda()
        self.fe = dict(flags=7, lower_bound=-5.0, l2_eps=1e-6, A_log=torch.zeros(H).cuda(),
                       dt_bias=torch.zeros(H, 128).cuda())
        self.conv_pool = torch.zeros(slots, 3, 3 * H * 128, dtype=torch.bfloat16).cuda()
        self.kda_pool = torch.zeros(slots, H, 128, 128).cuda()

    def _proj(self, x, res):
        import kda_chunked_recurrent_b200 as K
        h, res, _ = K.rms_norm(x, self.w1, residual=res)
        u = h @ self.gates
        n = H * 128
        a = u[:, :n].contiguous().view(-1, H, 128)
        return h @ self.qkv, a, u[:, n:2 * n].unflatten(1, (H, 128)), u[:, 2 * n:].contiguous(), res

    def _end(self, o, z, res):
        import kda_chunked_recurrent_b200 as K
        q, _, s = K.rms_norm(o, self.w2, gate=z, gate_activation="sigmoid",
                             out_dtype=torch.float8_e4m3fn, group=128)
        y = (q.float() * s).bfloat16().flatten(1)
        return y @ self.out, res

    def prompts(self, x, res, cu, slots, has):
        import kda_chunked_recurrent_b200 as K
        u, a, z, beta, res = self._proj(x, res)
        qkv = K.conv_prefill(u, self.conv, state=self.conv_pool, state_indices=slots, has_state=has,
                             cu_seqlens=cu, parts=3).unflatten(2, (H, 128))
        h0 = self.kda_pool[slots.long()] * has[:, None, None, None]
        o, ht, _ = K.prefill(qkv[0], qkv[1], qkv[2], a, beta, 128 ** -0.5, h0=h0, cu_seqlens=cu,
                             frontend=self.fe)
        self.kda_pool[slots.long()] = ht
        return self._end(o, z, res)

    def tokens(self, x, res, slots, T):
        import kda_chunked_recurrent_b200 as K
        u, a, z, beta, res = self._proj(x, res)
        f = lambda v: v.unflatten(0, (-1, T))  # noqa: E731
        qkv, _ = K.conv_decode(f(u), self.conv, self.conv_pool, state_indices=slots, parts=3)
        q, k, v = qkv.unflatten(3, (H, 128))
        o, _ = K.decode(q, k, v, f(a), f(beta), 128 ** -0.5, self.kda_pool, state_indices=slots,
                        frontend=self.fe)
        return self._end(o.flatten(0, 1), z, res)


def _relative(a, b):
    return float((a.float() - b.float()).norm() / b.float().norm())


def test_kda_layer_prompts_then_tokens_follow_one_prompt():
    """Two requests: prompts of 70 and 33 rows, two drafts each, then three tokens each, against
    whole prompts of 75 and 38 rows.  Rows are BF16 and pass an E4M3 rounding (2^-4) and BF16
    products, and a value next to a rounding border may go to the other side: 2-norm of the
    difference of two such roundings."""
    g = torch.Generator().manual_seed(1)
    lens, more = [70, 33], 5
    xs = [torch.randn(n + more, DM, generator=g).bfloat16().cuda() for n in lens]
    rs = [torch.randn(n + more, DM, generator=g).bfloat16().cuda() for n in lens]
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    cold = torch.zeros(2, dtype=torch.bool, device="cuda")
    cu = lambda ns: torch.tensor([0, ns[0], ns[0] + ns[1]], dtype=torch.int32, device="cuda")  # noqa: E731

    whole = KdaLayer(3)
    y, r = whole.prompts(torch.cat(xs), torch.cat(rs), cu([n + more for n in lens]), slots, cold)
    want = [y[:lens[0] + more], y[lens[0] + more:]]

    layer = KdaLayer(3)
    part = lambda v, a, b: torch.cat([t[n + a:n + b] for t, n in zip(v, lens)])  # noqa: E731
    y, r = layer.prompts(torch.cat([t[:n] for t, n in zip(xs, lens)]),
                         torch.cat([t[:n] for t, n in zip(rs, lens)]), cu(lens), slots, cold)
    got = [[y[:lens[0]]], [y[lens[0]:]]]
    for a, b in [(0, 2), (2, 3), (3, 4), (4, 5)]:
        y, r = layer.tokens(part(xs, a, b), part(rs, a, b), slots, b - a)
        for i, v in enumerate(y.unflatten(0, (2, -1))):
            got[i].append(v)
    for i in range(2):
        assert _relative(torch.cat(got[i]), want[i]) < 2 * 2.0 ** -4
        tail = slice(lens[i], None)
        assert _relative(torch.cat(got[i])[tail], want[i][tail]) < 2 * 2.0 ** -4
    assert torch.equal(layer.conv_pool[[2, 0]], whole.conv_pool[[2, 0]])
    # the recurrence's own tolerance, once per side
    assert _relative(layer.kda_pool[[2, 0]], whole.kda_pool[[2, 0]]) < 2e-3
    assert torch.all(layer.conv_pool[1] == 0) and torch.all(layer.kda_pool[1] == 0)


class ScanLayer:
    """norm -> x, z -> short convolution -> selective scan (gated) -> output"""
    D, S = 192, 16

    def __init__(self, slots, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: (torch.randn(*s, generator=g) * s[0] ** -0.5).bfloat16().cuda()  # noqa: E731
        D, S = self.D, self.S
        self.win, self.wx, self.wdt, self.wout = r(DM, 2 * D), r(D, 8 + 2 * S), r(8, D), r(D, DM)
        self.conv, self.bias = torch.randn(D, 4, generator=g).cuda(), torch.randn(D, generator=g).cuda()
        self.A_log = torch.log(torch.arange(1, S + 1).float()).repeat(D, 1).cuda()
        self.skip, self.dt_bias = torch.ones(D).cuda(), torch.full((D,), -4.0).cuda()
        self.conv_pool = torch.zeros(slots, 3, D, dtype=torch.bfloat16).cuda()
        self.pool = torch.zeros(slots, D, S).cuda()

    def run(self, x, conv, scan):
        import kda_chunked_recurrent_b200 as K
        D, S = self.D, self.S
        xz = K.rms_norm(x)[0] @ self.win
        u = conv(xz[:, :D])
        low = u @ self.wx
        dt = low[:, :8] @ self.wdt
        B, C = low[:, 8:8 + S].unflatten(1, (1, S)), low[:, 8 + S:].unflatten(1, (1, S))
        return scan(u, dt, B, C, xz[:, D:]) @ self.wout

    def prompts(self, x, cu, slots, has):
        import kda_chunked_recurrent_b200 as K
        kw = dict(state_indices=slots, has_state=has, cu_seqlens=cu)
        return self.run(
            x, lambda u: K.conv_prefill(u, self.conv, bias=self.bias, state=self.conv_pool, **kw),
            lambda u, dt, B, C, z: K.scan_prefill(u, dt, self.A_log, B, C, D=self.skip, z=z,
                                                  dt_bias=self.dt_bias, state=self.pool, **kw))

    def tokens(self, x, slots, T):
        import kda_chunked_recurrent_b200 as K
        f = lambda v: v.unflatten(0, (-1, T))  # noqa: E731
        return self.run(
            x, lambda u: K.conv_decode(f(u), self.conv, self.conv_pool, bias=self.bias,
                                       state_indices=slots)[0].flatten(0, 1),
            lambda u, dt, B, C, z: K.scan_decode(
                f(u), f(dt), self.A_log, f(B), f(C), self.pool, D=self.skip, z=f(z),
                dt_bias=self.dt_bias, state_indices=slots)[0].flatten(0, 1))


def test_scan_layer_prompts_in_pieces_then_tokens_follow_one_prompt():
    """Chunked prompts (the second chunk continues from the slots) and tokens against whole
    prompts; the products around the operators are the same rows in other batches, so rows may
    differ by BF16 roundings that fall on the other side: a few of 2^-8."""
    g = torch.Generator().manual_seed(2)
    lens = [60, 41]
    xs = [torch.randn(n, DM, generator=g).bfloat16().cuda() for n in lens]
    slots = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    cold, warm = (torch.full((2,), v, dtype=torch.bool, device="cuda") for v in (False, True))
    cu = lambda *c: torch.tensor(c, dtype=torch.int32, device="cuda")  # noqa: E731
    whole = ScanLayer(4)
    y = whole.prompts(torch.cat(xs), cu(0, 60, 101), slots, cold)
    layer = ScanLayer(4)
    got = [[], []]
    a = layer.prompts(torch.cat([xs[0][:33], xs[1][:2]]), cu(0, 33, 35), slots, cold)
    got[0].append(a[:33]), got[1].append(a[33:])
    a = layer.prompts(torch.cat([xs[0][33:55], xs[1][2:36]]), cu(0, 22, 56), slots, warm)
    got[0].append(a[:22]), got[1].append(a[22:])
    for lo, hi in [(0, 3), (3, 4), (4, 5)]:
        a = layer.tokens(torch.cat([xs[0][55 + lo:55 + hi], xs[1][36 + lo:36 + hi]]), slots, hi - lo)
        got[0].append(a[:hi - lo]), got[1].append(a[hi - lo:])
    for g_, w in zip(got, (y[:60], y[60:])):
        assert _relative(torch.cat(g_), w) < 4 * 2.0 ** -8
    assert _relative(layer.pool, whole.pool) < 4 * 2.0 ** -8
    assert _relative(layer.conv_pool, whole.conv_pool) < 4 * 2.0 ** -8


def _token_step(layer, x, slots):
    return layer.tokens(x, slots, 1)


def test_captured_step_replays_with_new_rows():
    """A decode step of the whole layer captured once and replayed: the rows, slots and pools
    are read at replay."""
    g = torch.Generator().manual_seed(3)
    x = [torch.randn(4, DM, generator=g).bfloat16().cuda() for _ in range(3)]
    sl = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 3, 2, 1], [4, 1, -1, 0],
                                                                     [2, 5, 1, 0])]
    eager, graphed = ScanLayer(6), ScanLayer(6)
    want = [_token_step(eager, a, s) for a, s in zip(x, sl)]
    xin, sin = x[0].clone(), sl[0].clone()
    warm = ScanLayer(6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _token_step(warm, xin, sin)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _token_step(graphed, xin, sin)
    for a, s, w in zip(x, sl, want):
        xin.copy_(a)
        sin.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert torch.equal(graphed.pool, eager.pool)
    assert torch.equal(graphed.conv_pool, eager.conv_pool)


def test_captured_prompts_replay_with_new_lengths():
    """A padded prompt batch captured once: the offsets are read at replay, rows behind the last
    sequence stay as they were."""
    import kda_chunked_recurrent_b200 as K
    g = torch.Generator().manual_seed(4)
    x = torch.randn(64, 96, generator=g).bfloat16().cuda()
    w = torch.randn(96, 4, generator=g).cuda()
    A_log, dt_bias = torch.zeros(96, 16).cuda(), torch.full((96,), -3.0).cuda()
    BC = torch.randn(64, 2, 1, 16, generator=g).bfloat16().cuda()
    cu = torch.tensor([0, 20, 64], dtype=torch.int32, device="cuda")
    out, y = torch.empty_like(x), torch.empty_like(x)

    def step():
        K.conv_prefill(x, w, cu_seqlens=cu, out=out)
        K.scan_prefill(out, x, A_log, BC[:, 0], BC[:, 1], dt_bias=dt_bias, cu_seqlens=cu, out=y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for offsets in ([0, 20, 64], [0, 7, 50], [0, 0, 33]):
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        out.fill_(5)
        y.fill_(6)
        graph.replay()
        torch.cuda.synchronize()
        o, z = out.clone(), y.clone()
        out.fill_(5)
        y.fill_(6)
        step()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(z, y)
        assert torch.all(o[offsets[2]:] == 5) and torch.all(z[offsets[2]:] == 6)


def test_calls_on_their_own_streams():
    """Calls on several streams at once give what they give one after the other."""
    g = torch.Generator().manual_seed(5)
    x = [torch.randn(200, DM, generator=g).bfloat16().cuda() for _ in range(3)]
    cu = torch.tensor([0, 150, 200], dtype=torch.int32, device="cuda")
    sl = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    cold = torch.zeros(2, dtype=torch.bool, device="cuda")
    want, pools = [], []
    for a in x:
        layer = ScanLayer(2)
        want.append(layer.prompts(a, cu, sl, cold))
        pools.append(layer.pool)
    layers = [ScanLayer(2) for _ in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    got = []
    for layer, a, s in zip(layers, x, streams):
        with torch.cuda.stream(s):
            got.append(layer.prompts(a, cu, sl, cold))
    torch.cuda.synchronize()
    for layer, a, b, p in zip(layers, got, want, pools):
        assert torch.equal(a, b) and torch.equal(layer.pool, p)


def test_an_explicit_stream_is_used():
    import kda_chunked_recurrent_b200 as K
    s = torch.cuda.Stream()
    x = torch.randn(64, 256, device="cuda")
    want = K.rms_norm(x)[0]
    torch.cuda.synchronize()
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    # captured on s: a launch that went to another stream would not be in the graph
    with torch.cuda.graph(graph, stream=s):
        K.rms_norm(x, out=out, stream=s)
    torch.cuda.synchronize()
    assert torch.all(out == 0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("call", [
    lambda K, x, w, s: K.rms_norm(x, stream=s)[0],
    lambda K, x, w, s: K.conv_prefill(x, w, stream=s),
], ids=["norm", "conv"])
def test_outputs_belong_to_the_given_stream(call):
    """An output is not memory that the current stream has just freed: its work there, which the
    given stream does not wait for, may not be done."""
    import kda_chunked_recurrent_b200 as K
    s = torch.cuda.Stream()
    x = torch.randn(4099, 1031, device="cuda")     # a size that nothing else has
    w = torch.ones(1031, 4, device="cuda")
    torch.cuda.synchronize()
    freed = torch.empty_like(x)
    address = freed.data_ptr()
    del freed
    again = torch.empty_like(x)
    assert again.data_ptr() == address             # so the allocator gives it out again
    del again
    other = call(K, x, w, s)
    torch.cuda.synchronize()
    assert other.data_ptr() != address
    with torch.cuda.stream(s):
        same = call(K, x, w, None)
    torch.cuda.synchronize()
    assert torch.equal(other, same)
