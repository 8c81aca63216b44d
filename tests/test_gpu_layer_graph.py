"""The layer operators captured in HIP graphs, with eager work and synchronisation between the replays: the results
must be the eager ones bit for bit, also where two graphs share a workspace."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _randn(*shape, dtype=torch.float32, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed + sum(shape))).to("cuda", dtype)


def _capture(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    return graph


def _replays(calls, results, before=lambda: None):
    """Each of `calls` writes its tensors of `results`; captures each and checks four replays of all in turn.
    before() puts back what the calls work on in place."""
    want = []
    for call, out in zip(calls, results):
        before()
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
    graphs = [_capture(call) for call in calls]
    for rep in range(4):
        for graph, out, w in zip(graphs, results, want):
            for t in out:
                t.zero_()
            before()
            torch.cuda.synchronize()
            graph.replay()
            _ = torch.ones(1000, device="cuda").sum().item()
            torch.cuda.synchronize()
            for t, v in zip(out, w):
                assert torch.equal(t, v), rep


def test_graph_replays_of_the_convolution():
    import selective_state_space_22_amd as lib

    bf, shape = torch.bfloat16, (3, 700, 260)
    x, dout, w, bias = _randn(*shape, dtype=bf), _randn(*shape, dtype=bf, seed=1), _randn(260, 4), _randn(260)
    reset = torch.rand(3, 700, generator=torch.Generator().manual_seed(0)).cuda() < 0.01
    n = torch.tensor([700, 0, 333], dtype=torch.int32, device="cuda")
    out, last = torch.empty_like(x), torch.empty((3, 3, 260), dtype=bf, device="cuda")
    g = {"dx": torch.empty_like(x), "dweight": torch.empty_like(w), "dbias": torch.empty_like(bias),
         "dwindow": torch.empty_like(last)}
    ws = torch.empty(lib.mamba_conv_bwd_workspace_size(*shape, 4, lib.MAMBA_IO_BF16), dtype=torch.uint8, device="cuda")
    g2 = {k: torch.empty_like(v) for k, v in g.items()}
    _replays([lambda: lib.mamba_conv_fwd(x, w, bias=bias, reset=reset, lengths=n, out=out, last_window=last),
              lambda: lib.mamba_conv_bwd(x, w, dout, bias=bias, reset=reset, grads=g, workspace=ws),
              lambda: lib.mamba_conv_bwd(dout, w, x, bias=bias, grads=g2, workspace=ws)],
             [[out, last], list(g.values()), list(g2.values())])


@pytest.mark.parametrize("batch", [2, 40])
def test_graph_replays_of_a_token(batch):
    import selective_state_space_22_amd as lib

    bf, D, N, R = torch.bfloat16, 200, 16, 13
    x, z, cw, A = _randn(batch, D, dtype=bf), _randn(batch, D, dtype=bf, seed=1), _randn(D, 4), -_randn(D, N).abs()
    Wx, Wdt = _randn(R + 2 * N, D, dtype=bf), _randn(D, R, dtype=bf)
    state0, window0 = _randn(2 * batch, D, N), _randn(2 * batch, 3, D, dtype=bf)
    state, window = state0.clone(), window0.clone()
    slots = torch.randperm(2 * batch, generator=torch.Generator().manual_seed(0))[:batch].to("cuda", torch.int32)
    slots[-1] = -1
    out, cout = torch.zeros_like(x), torch.zeros_like(x)
    ws = torch.empty(lib.mamba_conv_ssm_update_workspace_size(batch, D, N, R, lib.MAMBA_IO_BF16), dtype=torch.uint8,
                     device="cuda")

    def before():
        state.copy_(state0)
        window.copy_(window0)

    _replays([lambda: lib.mamba_conv_ssm_update(state, window, x, cw, Wx, Wdt, A, z=z, slots=slots, out=out, workspace=ws),
              lambda: lib.mamba_conv_ssm_update(state, window, z, cw, Wx, Wdt, A, slots=slots, out=cout, workspace=ws),
              lambda: lib.mamba_conv_update(window, x, cw, slots=slots, out=cout)],
             [[out, state, window], [cout, state, window], [cout, window]], before)


@pytest.mark.parametrize("shape", [(900, 768), (70, 5000)], ids=str)
def test_graph_replays_of_the_norms(shape):
    import selective_state_space_22_amd as lib

    bf, D = torch.bfloat16, shape[1]
    x, gate, dout = (_randn(*shape, dtype=bf, seed=s) for s in range(3))
    res, dres = _randn(*shape, seed=4), _randn(*shape, seed=5)
    pre, post, scale = (_randn(D, seed=s) for s in range(3))
    out, rout = torch.empty_like(x), torch.empty_like(res)
    part = {"gate": gate, "post_weight": post, "scale": scale, "residual": res}
    g = {"dx": torch.empty_like(x), "dgate": torch.empty_like(x), "dresidual": torch.empty_like(res),
         "dpost_weight": torch.empty_like(pre), "dscale": torch.empty_like(pre), "dpre_weight": torch.empty_like(pre)}
    ws = torch.empty(lib.mamba_residual_norm_bwd_workspace_size(*shape, lib.MAMBA_IO_BF16), dtype=torch.uint8, device="cuda")
    _replays([lambda: lib.mamba_residual_norm_fwd(x, pre, out=out, residual_out=rout, **part),
              lambda: lib.mamba_residual_norm_bwd(x, pre, dout, dresidual_out=dres, grads=g, workspace=ws, **part)],
             [[out, rout], list(g.values())])


@pytest.mark.parametrize("rows,K,V", [(1, 3, 30000), (50, 2, 1000)])
def test_graph_replays_of_the_verification(rows, K, V):
    import selective_state_space_22_amd as lib

    p, q = torch.softmax(_randn(rows, K + 1, V), -1), torch.softmax(_randn(rows, K, V, seed=1), -1)
    ids = torch.randint(0, V, (rows, K), generator=torch.Generator().manual_seed(0)).cuda()
    u, noise = torch.rand((rows, K), device="cuda"), torch.empty((rows, V), device="cuda").exponential_()
    tokens = torch.empty((rows, K + 1), dtype=torch.int64, device="cuda")
    kept = torch.empty((rows,), dtype=torch.int32, device="cuda")
    ws = torch.empty(lib.mamba_draft_verify_workspace_size(rows, K, V, 0) + 1, dtype=torch.uint8, device="cuda")
    _replays([lambda: lib.mamba_draft_verify(p, q, ids, u, noise, tokens=tokens, accepted=kept, workspace=ws)],
             [[tokens, kept]])
