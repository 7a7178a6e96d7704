"""The operators together: the example trains a small descriptor network and matches with it."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_training_lowers_the_loss_and_matches():
    """Untrained, descriptors are mostly noise and a match's loss is above the logarithm of the matches' number (log 340 = 5.8);
    trained, an unseen pair's reciprocal matches are mostly true ones."""
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_descriptors.py")
    spec = importlib.util.spec_from_file_location("train_descriptors", at)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    first, last, share, found = m.train(steps=60, log=lambda *a: None)
    assert last < 0.5 * first
    assert found >= 30 and share > 0.7
