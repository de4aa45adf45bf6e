"""What a dropout object and a program's dropout op are told and refuse, without a GPU."""
import pytest

from gemm_epilogue_transformer_smem_gb300 import api, build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


@pytest.mark.parametrize("dropout", [None, 0.5])
@pytest.mark.parametrize("spec", ["dropout:0.1", "dropout:0"])
def test_the_op_takes_no_number(spec, dropout):
    """The probability is the object's: a number behind the op would be ignored, and the op with it."""
    rng = None if dropout is None else api.Dropout(dropout, device="cpu")
    with pytest.raises(ValueError):
        api.Plan(64, 64, 64, [spec, "store_bf16"], b_layout="nk", dropout=rng)


@pytest.mark.parametrize("name,value", [("p", 0.0), ("threshold", 0)])
def test_the_probability_stays(name, value):
    """Plans hold it: one that changed later would give masks of two probabilities for one step."""
    rng = api.Dropout(0.5, device="cpu")
    with pytest.raises(AttributeError):
        setattr(rng, name, value)
    assert rng.p == 0.5 and rng.threshold == 32768
    assert api._mask(rng, 3, -1) == (rng.step.data_ptr(), 0, 3, 32768)
