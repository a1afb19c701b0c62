"""What K2_OPT_ACT8 costs those who do not use it: nothing of the workspace.  No GPU is needed."""
import pytest

import k2_inputs as ki


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import build
    build.build()
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


def grows(k2, **sizes):
    """Workspace bytes that a row more of a size takes."""
    (name, n), = sizes.items()
    make = lambda v: k2.workspace_bytes(k2.make_config(ki.K2_3P7B.replace(**{name: v}), 4096, weights="f8"))  # noqa: E731
    return (make(2 * n) - make(n)) / n


def test_the_workspace_of_an_fp8_model_holds_no_copies_for_it(k2):
    s = ki.K2_3P7B
    # a row of the vocabulary: its codes; a scale, logits and candidates of some sequences and of a verification
    assert s.hidden <= grows(k2, vocab=s.vocab) < 1.1 * s.hidden
    # a gate, its factor and a column of down: codes, and those as bf16, in each layer; rows of a prefill block
    assert 9 * s.hidden * s.n_layers <= grows(k2, intermediate=s.intermediate) < 9.3 * s.hidden * s.n_layers


def test_calls_on_no_context(k2):
    assert k2.LIB.k2_act8_bytes(None) == 0
    assert k2.LIB.k2_act8_init(None, None, 0, None) == k2.K2_ERR_ARG
