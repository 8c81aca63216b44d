"""The token-model operators captured in a HIP graph, with eager work and synchronisation between the
replays: the results must be the eager ones bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _randn(*shape, dtype=torch.float32, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed + sum(shape))).to("cuda", dtype)


def _replays(call, results):
    """call() writes the tensors `results`; captures it and checks four replays."""
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in results]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for rep in range(4):
        for t in results:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(results, want):
            assert torch.equal(t, w), rep
        _ = (want[0].float() * 2).sum().item()


@pytest.mark.parametrize("shape", [(1, 20000, 64), (3, 1500, 520)], ids=str)
def test_graph_replays_of_the_gated_scan(shape):
    import selective_state_space_22_amd as lib

    batch, L, D = shape
    bf = torch.bfloat16
    u, a, x, z, dout = (_randn(*shape, dtype=bf, seed=s) for s in range(5))
    lam = _randn(D) - 5.0
    out, last = torch.empty_like(u), torch.empty((batch, D), device="cuda")
    states = torch.empty((batch, -(-L // lib.MAMBA_GATED_STATE_CHUNK), D), device="cuda")
    ws = torch.empty(lib.mamba_gated_scan_fwd_workspace_size(*shape, lib.MAMBA_IO_BF16) + 1, dtype=torch.uint8,
                     device="cuda")
    _replays(lambda: lib.mamba_gated_scan_fwd(u, a, x, lam, z=z, out=out, last_state=last, states=states, workspace=ws),
             [out, last, states])
    g = {k: torch.empty_like(u) for k in ("du", "dgate_a", "dgate_x", "dz")}
    g.update(dlam=torch.empty_like(lam), dh0=torch.empty_like(last))
    wb = torch.empty(lib.mamba_gated_scan_bwd_workspace_size(*shape, lib.MAMBA_IO_BF16) + 1, dtype=torch.uint8,
                     device="cuda")
    _replays(lambda: lib.mamba_gated_scan_bwd(u, a, x, lam, dout, z=z, states=states, grads=g, workspace=wb),
             list(g.values()))


@pytest.mark.parametrize("count", [500, 9000])
def test_graph_replays_of_a_table_gradient(count):
    import selective_state_space_22_amd as lib

    ids = torch.randint(-1, 700, (count,), generator=torch.Generator().manual_seed(2)).cuda()
    dout, dw = _randn(count, 72), torch.empty((700, 72), device="cuda")
    ws = torch.empty(lib.mamba_embed_bwd_workspace_size(count, 700, 72, lib.MAMBA_IO_F32) + 1, dtype=torch.uint8,
                     device="cuda")
    _replays(lambda: lib.mamba_embed_bwd(ids, dout, 700, dweight=dw, workspace=ws), [dw])


def test_graph_replays_of_a_generated_token():
    import selective_state_space_22_amd as lib

    V, D, B = 5003, 256, 4
    table, lam, start = _randn(V, D), _randn(D) - 5.0, _randn(B, D, seed=1)
    ids = torch.tensor([5, 4000, 77, 5002], device="cuda")
    noise = torch.rand((B, V), generator=torch.Generator().manual_seed(3)).cuda() + 0.1
    top_p, state = torch.full((B,), 0.9, device="cuda"), torch.empty_like(start)
    x, y = torch.empty((B, D), device="cuda"), torch.empty((B, D), device="cuda")
    token, logprob = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(B, device="cuda")
    logits = _randn(B, V, seed=4)

    def call():
        state.copy_(start)
        lib.mamba_embed_fwd(ids, table, out=x)
        lib.mamba_gated_state_update(state, x, x, x, lam, z=x, out=y)
        lib.mamba_sample(logits, noise, top_p=top_p, tokens=token, logprob=logprob)

    _replays(call, [x, state, y, token, logprob])
