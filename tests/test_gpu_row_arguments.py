"""Calls that are refused before any launch, the short way (no stream given) and the
way through Python (a stream given) alike."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sigmoid_top_routing_router_amd as M
    M.load_library()
    return M


def both_ways(call, kind, match):
    import torch
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(kind, match=match):
            call(stream)


@pytest.mark.parametrize("d", [1, 64, 127, 192])
def test_codes_of_rows_without_whole_groups(M, d):
    import torch

    def kept(n):
        return (torch.zeros(n, d, dtype=torch.uint8, device="cuda"),
                torch.zeros(n, d // 128, device="cuda"))
    g = M.group_tokens(torch.tensor([[0, 1], [1, 2], [2, 0]], dtype=torch.int32, device="cuda"), 3)
    dy = torch.zeros(3, d, dtype=torch.bfloat16, device="cuda")
    both_ways(lambda s: M.permute(kept(3), g, stream=s), M.MoeError, "multiple of 128")
    both_ways(lambda s: M.unpermute_backward(dy, g, rows=kept(6), stream=s), M.MoeError,
              "multiple of 128")
    rows = torch.zeros(6, d, dtype=torch.bfloat16, device="cuda")
    both_ways(lambda s: M.unpermute(rows, g, checkpoint=True, stream=s), M.MoeError,
              "multiple of 128")


def test_a_grouping_without_tensors_is_no_dense_product(M):
    import torch
    q = torch.zeros(4, 32, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    w = torch.zeros(8, 32, dtype=torch.int8, device="cuda"), torch.zeros(8, device="cuda")
    none = M.Grouping(None, None, None, None)
    both_ways(lambda s: M.int8_matmul(q, w, grouping=none, stream=s), ValueError, "expected")
    both_ways(lambda s: M.int8_matmul(q, (w[0][None], w[1][None]), grouping=none, stream=s),
              ValueError, "src_pos must be")


def test_a_workspace_elsewhere_or_expanded(M):
    import torch
    N, d, E, K, h = 4, 64, 3, 2, 32
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")
    x, logits, ids = z(N, d), z(N, E, t=torch.float32), z(N, K, t=torch.int32)
    W = M.ExpertWeights(w_router=z(E, d), w_gate=z(E, h, d), w_up=z(E, h, d), w_down=z(E, d, h))
    calls = (lambda ws, s: M.eqb_bias(logits, K, workspace=ws, stream=s),
             lambda ws, s: M.forward(x, W, K, workspace=ws, stream=s),
             lambda ws, s: M.backward(x, x, W, logits, ids, workspace=ws, stream=s),
             lambda ws, s: M.rms_norm_backward(x, x, z(d), workspace=ws, stream=s),
             lambda ws, s: M.balance_loss(logits, ids, workspace=ws, stream=s),
             lambda ws, s: M.group_tokens(ids, E, workspace=ws, stream=s))
    for call in calls:
        both_ways(lambda s: call(torch.zeros(1 << 20, dtype=torch.uint8), s), ValueError,
                  "workspace is on cpu")
        both_ways(lambda s: call(z(256, t=torch.uint8)[:1].expand(1 << 20), s), ValueError,
                  "workspace must be contiguous")
