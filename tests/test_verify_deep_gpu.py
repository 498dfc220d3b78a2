"""Chains of which many drafts are kept, over large vocabularies: batches that
walk and batches whose rows are drawn from at once, each sequence to a depth of
its own, the last node among them."""
import pytest
import torch

from rank_adapter_gemm_token_amd import lora

pytestmark = pytest.mark.gpu

I = dict(dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("seqs,nodes,vocab,dtype", [
    (128, 32, 131072, torch.bfloat16), (40, 32, 131072, torch.bfloat16), (64, 32, 32000, torch.float32),
    (16, 32, 32000, torch.float32), (1, 63, 131072, torch.float16), (250, 20, 5001, torch.float32)])
def test_kept_to_every_depth(seqs, nodes, vocab, dtype):
    R = seqs * nodes
    kept = torch.arange(seqs, device="cuda") * 7 % nodes if seqs > 1 else torch.tensor([nodes - 1], device="cuda")
    node = torch.arange(nodes, device="cuda").expand(seqs, nodes)
    # At node i the next node's token is drawn as long as i is below the depth,
    # then one that no child holds: each is likelier than all others together.
    token = torch.where(node < kept[:, None], 200 + node + 1, vocab - 1 - node)
    p = torch.full((R, vocab), 1e-6, dtype=dtype, device="cuda")
    p.scatter_(1, token.reshape(R, 1), 1.0)
    draft, parent = (200 + node).reshape(R).int(), (node - 1).reshape(R).int()
    row0 = torch.arange(0, R + 1, nodes, **I)
    tokens, path, accepted = (torch.full((n,), -7, **I) for n in (R, R, seqs))
    v = lora.lora_verifier_create(seqs)
    lora.lora_verify_tree(v, p, draft, parent, row0, torch.full((R,), 0.5, device="cuda"), seqs, R, tokens, path, accepted)
    on = node <= kept[:, None]
    assert torch.equal(accepted.long(), kept)
    assert torch.equal(tokens.view(seqs, nodes).long(), torch.where(on, token, -1))
    assert torch.equal(path.view(seqs, nodes).long(), torch.where(on, node, -1))
    lora.lora_verifier_destroy(v)
