"""Training sublayer on dense gates: every row has more active neurons than a
sparse row holds, so all of them live in the dense backup."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def block():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import block as mod

    return mod


def dense(M=200, K=256, N=1024):
    """Inputs at random initialisation: about half of the N neurons of every
    row are active, four times the 128 entries of a sparse row."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=g)
    gamma, beta = 1 + 0.1 * torch.randn(K, generator=g), 0.1 * torch.randn(K, generator=g)
    w = [(torch.randn(N, K, generator=g) * s).bfloat16() for s in (K ** -0.5, K ** -0.5, N ** -0.5)]
    return x, gamma, beta, *w


def fill_free_memory():
    """NaN in the blocks that the allocator will hand out next."""
    for shape in ((200, 256), (200, 256), (200, 1024), (400, 1024)):
        torch.full(shape, float("nan"), device="cuda")


def off(a, b):
    return ((a.double().cpu() - b).norm() / b.norm()).item()


def test_default_capacity_holds_every_row(block):
    """y and every gradient against float64, at the default arguments.  The
    norm's output, the gradient of y and the backup are bf16 (2^-8 each), every
    sum fp32: under 2 per cent."""
    args = dense()
    wide = [t.double().requires_grad_() for t in args]
    ref = block._reference(*wide)
    dy = torch.randn(200, 256, generator=torch.Generator().manual_seed(2))
    (ref * dy).sum().backward()
    fill_free_memory()
    y, saved = block.train_forward(*(t.cuda() for t in args))
    assert int(saved["hy"]["bk_count"]) == 200, "every row is to need the backup"
    assert off(y, ref.detach()) < 0.02
    fill_free_memory()
    got = block.train_backward(dy.cuda(), saved)
    for k, t in zip(("dx", "dgamma", "dbeta", "dwg_t", "dwu_t", "dwd"), wide):
        assert off(got[k], t.grad) < 0.02, k


@pytest.mark.parametrize("R_max", [0, 1, 199])
def test_too_small_a_backup_is_refused(block, R_max):
    """A row in neither store would have no output: the call says how many
    rows it needs."""
    with pytest.raises(RuntimeError, match="200 rows"):
        block.train_forward(*(t.cuda() for t in dense()), R_max=R_max)


def test_a_smaller_backup_that_is_enough(block):
    """Gates of 1 in 32 neurons: no row needs the backup, and one of no rows
    gives what one of every row gives."""
    x, gamma, beta, wg, wu, wd = dense()
    wg[32:] = 0
    args = [t.cuda() for t in (x, gamma, beta, wg, wu, wd)]
    y, saved = block.train_forward(*args)
    y0, saved0 = block.train_forward(*args, R_max=0)
    assert torch.equal(y, y0) and int(saved["hy"]["bk_count"]) == 0
    dy = torch.randn(200, 256, generator=torch.Generator().manual_seed(2)).cuda()
    a, b = block.train_backward(dy, saved), block.train_backward(dy, saved0)
    for k in a:
        assert torch.equal(a[k], b[k]), k
