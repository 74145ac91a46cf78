"""Training of the routed experts at sizes that tests/test_gpu_train.py leaves out:
together every way in which its products are cut runs, as tests/test_train_cuts.py
checks against the plan."""
import pytest
import torch

from tests.test_gpu_train import Case

pytestmark = pytest.mark.gpu

# act, T, H, E, I, k; a tenth of the pairs is dropped
MORE = [
    ("bf16", 1, 768, 1, 352, 1), ("bf16", 1, 768, 65, 352, 1), ("bf16", 33, 768, 1, 32, 1),
    ("bf16", 19, 1024, 64, 32, 4), ("bf16", 8423, 128, 256, 32, 1), ("bf16", 702, 768, 65, 32, 3),
    ("bf16", 568, 128, 65, 512, 4), ("bf16", 501, 1152, 64, 32, 10), ("bf16", 1494, 2432, 2, 32, 2),
    ("bf16", 2023, 1280, 70, 32, 3), ("bf16", 1330, 128, 70, 608, 3), ("bf16", 3179, 384, 65, 32, 8),
    ("bf16", 90, 128, 16, 2944, 10), ("bf16", 13413, 1024, 2, 32, 2), ("bf16", 3993, 2816, 65, 32, 3),
    ("bf16", 6941, 2304, 70, 32, 2), ("bf16", 1030, 128, 66, 960, 10),
    ("bf16", 9987, 128, 128, 512, 3), ("f32", 1, 384, 65, 192, 1),
    ("f32", 34, 384, 1, 32, 1), ("f32", 16, 4224, 16, 32, 1), ("f32", 1125, 384, 65, 32, 2),
    ("f32", 328, 1024, 33, 32, 8), ("f32", 2664, 512, 66, 32, 2), ("f32", 4282, 128, 70, 288, 1),
    ("f32", 4225, 256, 65, 96, 3), ("f32", 859, 128, 33, 1536, 3), ("f32", 4066, 512, 66, 32, 8),
    ("f32", 1059, 128, 9, 2272, 2), ("f32", 11838, 640, 65, 96, 1), ("f32", 5187, 640, 66, 256, 1),
    ("f32", 1585, 768, 70, 96, 8), ("f32", 4486, 768, 8, 96, 3), ("f32", 12104, 256, 65, 384, 1),
    ("f32", 2070, 1536, 8, 384, 1), ("f32", 4071, 128, 65, 448, 8), ("f32", 758, 4352, 16, 224, 4),
    ("f32", 198, 4352, 8, 928, 4)]


@pytest.mark.parametrize("kept", ["act", "8bit"])
@pytest.mark.parametrize("act,T,H,E,I,k", MORE)
def test_other_cuts(act, T, H, E, I, k, kept):
    what = f"{T} {H} {E} {I} {k} {act} {kept}"
    print(what, flush=True)
    c = Case(T, H, E, I, k, act, kept, drop=0.1, seed=19)
    c.save()
    c.check_save(f"save {what}")
    c = Case(T, H, E, I, k, act, kept, kept == "8bit", drop=0.1, seed=19)
    c.fill_saved()
    c.backward()
    c.check_backward(f"backward {what}")
    first = {n: v.clone() for n, v in c.grads().items()}
    c.backward()
    assert all(torch.equal(v, first[n]) for n, v in c.grads().items())
