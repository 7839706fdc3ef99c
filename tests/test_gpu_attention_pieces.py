"""The window attention's hand-over of work pieces from one SM of a pair to the other:
many short pieces a pair, launched over and over, with and without a gap."""
import pytest

from test_gpu_attention_op import make_problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    dict(n=40, T=200, H=12, dh=64, L=40),      # 480 pieces of one key tile
    dict(n=16, T=300, H=16, dh=128, L=300),    # 512 of two, half of them tails
    dict(n=6, T=520, H=12, dh=32, L=16500),    # tails in two halves of the keys
], ids=lambda c: f"n{c['n']}T{c['T']}L{c['L']}")
def test_pieces_are_never_mixed_up(case):
    import torch
    from autoregressive_denoising_dit_gb300 import _psv as P

    pb = make_problem(**case)
    prob = P.AttnProblem(**{k: pb[k] for k in ("n", "T", "H", "dh", "L", "k_rows", "vt_cols")})
    q, k, vt = (torch.from_numpy(pb[x]).to("cuda", dtype=torch.bfloat16) for x in ("q", "k", "vt"))
    n = P.psv_attention_scratch_bytes(prob)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert scratch.data_ptr() % 256 == 0
    outs = [torch.full_like(q, float(i)) for i in range(2)]
    stream = torch.cuda.current_stream().cuda_stream

    def call(o):
        P.psv_attention(prob, q.data_ptr(), k.data_ptr(), vt.data_ptr(), o.data_ptr(), scratch.data_ptr(), n, stream)

    call(outs[0])
    torch.cuda.synchronize()
    # each sequence alone gives the same rows: no piece was done in another's place
    for b in (0, case["n"] - 1):
        one = P.AttnProblem(**{**{x: pb[x] for x in ("T", "H", "dh", "L", "k_rows", "vt_cols")}, "n": 1})
        T = case["T"]
        o = torch.zeros_like(q[:T])
        P.psv_attention(one, q[b * T:(b + 1) * T].data_ptr(), k[b].data_ptr(), vt[b].data_ptr(), o.data_ptr(),
                        scratch.data_ptr(), n, stream)
        assert torch.equal(o, outs[0][b * T:(b + 1) * T])
    for i in range(200):
        call(outs[1])
        if i % 2:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(*outs)
    assert int(scratch[:4].view(torch.int32).item()) == 0
