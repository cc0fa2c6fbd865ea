"""What a 4-bit weight format does to a layer and to the model's loss.

One linear layer W in front of a vocabulary head U, activations X with
outlier channels, targets drawn from the full-precision model itself.  The
layer is coded at about 4 bits per weight three ways:

  qamw       the QAM-W codec (K = 256), decoded to bf16, activations in bf16
  mxfp4      microscaled 4-bit weights and activations (qamw_mxfp4_matmul)
  mxfp4+rot  the same after the codec's rotation: (R X)(R W)^T = X W^T

and measured by the layer-output error of its weights, by the relative error
of its outputs as they are run, by the change of the loss, and by how much of
the loss's gradient in the layer's outputs it keeps.

    python examples/compare_formats.py [--tokens 512 --d-in 4096 --d 512 --vocab 32000]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vector_codebook_codec_amd as q  # noqa: E402

BLOCK, SIGN_SEED = 128, 7


def layer_forms(W, X):
    """{name: (decoded weights, what they approximate, its activations, outputs as run)}, all bf16 matrices."""
    forms = {}
    C = torch.from_numpy(q.load_codebook(256)).to(W.device)
    s, sigma, packed, rn = q.qamw_calibrate_encode(W, q.qamw_channel_rms(X), 0.5, BLOCK, SIGN_SEED, C,
                                                   plan=q.qamw_build_plan(C))
    W_hat = q.qamw_decode(packed, rn, W.shape[1], s, sigma, BLOCK, SIGN_SEED, C, out_dtype=torch.bfloat16)
    Xr = q.qamw_rotate_activations(X, s, BLOCK, SIGN_SEED)
    forms["qamw"] = W_hat, W, X, q.qamw_decode_matmul(Xr, packed, rn, sigma, C, out_dtype=torch.bfloat16)
    rotate = lambda A: q.qamw_rotate_activations(A, None, BLOCK, SIGN_SEED)  # noqa: E731
    for name, w, x in (("mxfp4", W, X), ("mxfp4+rot", rotate(W), rotate(X))):
        codes, scales, W_hat = q.qamw_mxfp4_quantize(w, values_dtype=torch.bfloat16)
        forms[name] = W_hat, w, x, q.qamw_mxfp4_matmul(x, codes, scales, out_dtype=torch.bfloat16)
    return forms


def compare(tokens, d_in, d, vocab, seed=0, device="cuda:0"):
    """Rows (name, layer-output error, output error, loss, loss change, gradient kept), full precision first."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device=device, generator=g)  # noqa: E731
    outlier = torch.where(torch.rand(d_in, device=device, generator=g) < 0.01, 20.0, 1.0)
    X = (rand(tokens, d_in) * outlier).bfloat16()
    W = (rand(d, d_in) / outlier.square().sum().sqrt()).bfloat16()
    U = (rand(vocab, d) * (3.0 / d ** 0.5)).bfloat16()
    Y = (X.float() @ W.float().t()).bfloat16()
    targets = torch.multinomial(torch.softmax(Y.float() @ U.float().t(), dim=1), 1, generator=g).squeeze(1)
    upstream = torch.full((tokens,), 1.0 / tokens, device=device)

    def loss_and_gradient(H):
        loss, lse = q.qamw_cross_entropy(H, U, targets)
        dH, _ = q.qamw_cross_entropy_grad(H, U, targets, lse, upstream, need_dW=False)
        return loss.double().mean().item(), dH.double()

    base, dY = loss_and_gradient(Y)
    rows = [("bf16", 0.0, 0.0, base, 0.0, 1.0)]
    energy = Y.double().square().sum().item()
    for name, (W_hat, w, x, H) in layer_forms(W, X).items():
        loss, dH = loss_and_gradient(H)
        rows.append((name, (q.qamw_output_error(x, w, W_hat).item() / energy) ** 0.5,
                     ((H.double() - Y.double()).square().sum().item() / energy) ** 0.5, loss, loss - base,
                     torch.nn.functional.cosine_similarity(dH.flatten(), dY.flatten(), dim=0).item()))
    return rows


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--d-in", type=int, default=4096)
    ap.add_argument("--d", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args(argv)
    rows = compare(a.tokens, a.d_in, a.d, a.vocab)
    print(f"{'format':10s} {'weights alone':>14s} {'as run':>10s} {'loss':>9s} {'change':>9s} {'gradient cosine':>16s}")
    for name, layer, out, loss, change, cos in rows:
        print(f"{name:10s} {layer:14.4f} {out:10.4f} {loss:9.4f} {change:+9.4f} {cos:16.4f}")
    return rows


if __name__ == "__main__":
    main()
